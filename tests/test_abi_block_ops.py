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


# ------------------------------------------------------ differential attention
def _attn(**kw):
    a = dict(batch=2, q_len=70, k_len=90, q_heads=4, kv_heads=2, d=16, dv=32, scale=0.25, dtype=torch.bfloat16)
    after = {k: kw.pop(k) for k in list(kw) if k in ("dtype_code", "lam_code")}
    a.update(kw)
    d = rib.diff_attn_desc(**a)
    if "dtype_code" in after:
        d.dtype = after["dtype_code"]
    if "lam_code" in after:
        d.lam_dtype = after["lam_code"]
    return ctypes.byref(d)


ATTN = [P] * 5 + [P, None, P, P, P, P, 1 << 30, None]               # q1, q2, k1, k2, v, lam, k_lens, o, o2, lse, ws, bytes, stream
ATTN_BWD = [P] * 5 + [P, None] + [P] * 10 + [P, 1 << 30, None]      # ..., o, o2, lse, dO, dq1, dq2, dk1, dk2, dv, dlam, ws, bytes, stream


@pytest.mark.parametrize("kw,st", [
    ({"batch": -1}, INVALID), ({"q_len": -1}, INVALID), ({"k_len": -1}, INVALID), ({"q_heads": 0}, INVALID), ({"kv_heads": 0}, INVALID),
    ({"kv_heads": 3}, INVALID), ({"d": 0}, INVALID), ({"dv": -8}, INVALID), ({"d": 12}, UNSUPPORTED), ({"d": 72}, UNSUPPORTED),
    ({"dv": 136}, UNSUPPORTED), ({"scale": 0.0}, INVALID), ({"scale": -1.0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"dtype_code": 1}, INVALID), ({"dtype_code": 7}, INVALID), ({"lam_code": 2}, INVALID),
    ({"window": 8}, INVALID), ({"width": 8}, INVALID), ({"window": -1, "width": 8}, INVALID), ({"window": 8, "width": 10}, INVALID),
    ({"window": 8, "width": 8, "k_len": 70}, INVALID), ({"window": 8, "width": 10, "k_len": 70, "causal": True}, INVALID),
    ({"window": 1025, "width": 10, "k_len": 70}, UNSUPPORTED), ({"q_len": 0x7FFFFFFF}, UNSUPPORTED), ({"q_heads": 130}, UNSUPPORTED),
    ({"batch": 1 << 30}, UNSUPPORTED), ({"k_len": 0x7FFFFFFF}, UNSUPPORTED),
    ({"q_stride": (4480, 64, 4)}, ALIGNMENT), ({"k_stride": (-8, 32, 16)}, ALIGNMENT), ({"o_stride": (0, 128, 32)}, UNSUPPORTED),
    ({"o_stride": (8960, 32, 32)}, INVALID), ({"k_stride": (2880, 1 << 32, 16)}, UNSUPPORTED),
], ids=str)
def test_diff_attention_descriptor_refusals(lib, kw, st):
    d = _attn(**kw)
    assert lib.rib_diff_attention(d, *ATTN) == st
    assert lib.rib_diff_attention_bwd(d, *ATTN_BWD) == st
    assert lib.rib_diff_attention_workspace_size(d) == 0
    assert lib.rib_diff_attention_bwd_workspace_size(d) == 0


def test_diff_attention_argument_refusals(lib):
    f = lambda d, a: lib.rib_diff_attention(d, *a)  # noqa: E731
    b = lambda d, a: lib.rib_diff_attention_bwd(d, *a)  # noqa: E731
    assert f(None, ATTN) == INVALID and b(None, ATTN_BWD) == INVALID
    for i in (0, 1, 2, 3, 4, 5, 7):
        assert f(_attn(), _with(ATTN, **{f"_{i}": None})) == INVALID, i
    for i in [0, 1, 2, 3, 4, 5] + list(range(7, 18)):
        assert b(_attn(), _with(ATTN_BWD, **{f"_{i}": None})) == INVALID, i
    for i in (0, 1, 2, 3, 4, 7, 8, 10):
        assert f(_attn(), _with(ATTN, **{f"_{i}": 264})) == ALIGNMENT, i
    for i in [0, 1, 2, 3, 4, 7, 8] + list(range(10, 16)) + [17]:
        assert b(_attn(), _with(ATTN_BWD, **{f"_{i}": 264})) == ALIGNMENT, i
    assert f(_attn(), _with(ATTN, _5=257)) == ALIGNMENT and f(_attn(), _with(ATTN, _6=258)) == ALIGNMENT
    assert f(_attn(lam_dtype=torch.float32), _with(ATTN, _5=258)) == ALIGNMENT
    assert b(_attn(), _with(ATTN_BWD, _9=258)) == ALIGNMENT and b(_attn(), _with(ATTN_BWD, _16=257)) == ALIGNMENT
    w = dict(window=8, width=10, k_len=70)
    assert f(_attn(**w), _with(ATTN, _6=P)) == INVALID and b(_attn(**w), _with(ATTN_BWD, _6=P)) == INVALID   # windows and lengths
    assert b(_attn(), _with(ATTN_BWD, _18=100)) == INVALID                                                   # workspace too small
    # gradients that would lie on one another
    for k in ("q_stride", "k_stride"):
        assert b(_attn(**{k: (64, 64, 16)}), ATTN_BWD) == INVALID
    assert b(_attn(v_stride=(5760, 32, 32)), ATTN_BWD) == INVALID
    long = dict(batch=1, q_len=1, k_len=100000)
    assert lib.rib_diff_attention_workspace_size(_attn(**long)) > 0
    assert f(_attn(**long), _with(ATTN, _10=None)) == INVALID and f(_attn(**long), _with(ATTN, _11=64)) == INVALID
    assert f(_attn(batch=0), [None] * 11 + [0, None]) == 0 and f(_attn(q_len=0), [None] * 11 + [0, None]) == 0


def test_diff_attention_workspace_sizes(lib):
    # 60 bytes a row of row constants, 64 rows a box, an even number of boxes a key head; two cells of 8x7 and 2x7 tokens an item
    assert rib.rib_diff_attention_bwd_workspace_size(_attn()._obj) == 2 * 2 * 4 * 64 * 60
    assert rib.rib_diff_attention_bwd_workspace_size(_attn(q_len=70, k_len=70, window=8, width=10)._obj) == 2 * 2 * 2 * 2 * 64 * 60
    assert rib.rib_diff_attention_workspace_size(_attn()._obj) == 0
    for kw in ({"batch": 0}, {"q_len": 0}, {"k_len": 0}):
        assert rib.rib_diff_attention_workspace_size(_attn(**kw)._obj) == 0


def test_diff_attention_binding_refusals():
    d = rib.diff_attn_desc(1, 4, 4, 2, 2, 16, 32, 0.25, torch.bfloat16)
    t = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rib.rib_diff_attention(d, t, t, t, t, t, t, o=t)          # host tensors
    with pytest.raises(ValueError):
        rib.diff_attn_desc(1, 4, 4, 2, 2, 16, 32, 0.25, torch.int32)
    with pytest.raises(ValueError):
        _lib._strided_arg("q1", t, (1, 4, 2, 16), None, d.dtype, 0)


def test_diff_attention_layout_follows_descriptor():
    # one descriptor used again after its fields change: the checks see the new sizes, strides and types
    d = rib.diff_attn_desc(1, 4, 6, 2, 1, 16, 32, 0.25, torch.bfloat16)
    first = _lib._diff_layout(d)
    assert first[1:] == (((1, 4, 2, 16), None), ((1, 6, 1, 16), None), ((1, 6, 1, 32), None), ((1, 4, 2, 32), None), d.dtype, d.lam_dtype, 2, 1, 16)
    assert _lib._diff_layout(d) is first
    d.q_len = 9
    d.q_stride[0], d.q_stride[1], d.q_stride[2] = 576, 64, 32
    d.dtype += 1
    now = _lib._diff_layout(d)
    assert now[1] == ((1, 9, 2, 16), (576, 64, 32)) and now[4] == ((1, 9, 2, 32), None) and now[5] == d.dtype and now[-1] == 36
    d.q_stride[1] = 96
    assert _lib._diff_layout(d)[1][1] == (576, 96, 32)


def test_diff_attention_backward_scale_range(lib):
    # below it the row constants of the backward leave the 16-bit type; refused before any pointer is used
    for dtype, bad, ok in ((torch.float16, 2.0 ** -27, 2.0 ** -26), (torch.bfloat16, 2.0 ** -101, 2.0 ** -100)):
        assert lib.rib_diff_attention_bwd(_attn(dtype=dtype, scale=bad), *ATTN_BWD) == UNSUPPORTED
        assert lib.rib_diff_attention_bwd(_attn(dtype=dtype, scale=ok), *_with(ATTN_BWD, _0=None)) == INVALID   # the next check


def test_diff_attention_scale_in_powers_of_two(lib):
    # a finite scale whose product with log2 e is not
    for scale, st in ((2.4e38, INVALID), (2.3e38, 0)):
        d = _attn(scale=scale, batch=0)
        assert lib.rib_diff_attention(d, *ATTN) == st


def test_a_descriptor_made_field_by_field(monkeypatch):
    # the first call of a process, with a descriptor that no helper made: its tensors have the descriptor's type
    monkeypatch.setattr(_lib, "_TORCH_CODE", {})
    t = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)
    assert _lib._strided_arg("q1", t, (1, 4, 2, 16), None, _lib.RIB_BF16, t.get_device()) == t.data_ptr()
    monkeypatch.setattr(_lib, "_TORCH_CODE", {})
    with pytest.raises(ValueError):
        _lib._strided_arg("q1", t, (1, 4, 2, 16), None, _lib.RIB_F16, t.get_device())


def test_row_shapes_of_the_binding():
    f = lambda shape, want, t=torch.float32: _lib._row_arg("x", torch.zeros(shape, dtype=t), want, _lib.RIB_F32, -1)  # noqa: E731
    for shape in ((6, 40), (240,), (2, 3, 40), (6, 1, 40)):
        assert f(shape, (6, 40))
    assert f((40,), (40,)) and f((1, 40), (40,)) and f((0, 40), (0, 40)) is not None
    for shape, want in (((40, 6), (6, 40)), ((7, 40), (6, 40)), ((5, 40), (6, 40)), ((241,), (6, 40)), ((41,), (40,)), ((40, 1), (40,)),
                        ((2, 40), (40,)), ((), (6, 40))):
        with pytest.raises(ValueError):
            f(shape, want)
    with pytest.raises(ValueError):
        f((6, 40), (6, 40), torch.bfloat16)
    with pytest.raises(ValueError):
        _lib._row_arg("x", torch.zeros(40, 6).t(), (6, 40), _lib.RIB_F32, -1)
    assert _lib._row_arg("x", None, (6, 40), _lib.RIB_F32, -1) is None


def test_splits_where_they_pay(lib):
    # 148 SMs, as without a device. Splitting these cost 2.2, 1.5 and 1.1 times the call without it ...
    n, m = rib.rib_diff_attention_workspace_size, rib.rib_diff_attention_bwd_workspace_size
    shape = lambda b, q, k, hq, hk, d, dv, **kw: rib.diff_attn_desc(b, q, k, hq, hk, d, dv, 0.25, torch.bfloat16, **kw)  # noqa: E731
    assert n(shape(1, 1024, 1024, 6, 6, 16, 32)) == 0 and n(shape(32, 1, 1024, 16, 4, 64, 128)) == 0
    assert m(shape(1, 4096, 4096, 4, 4, 64, 128)) == 4 * 64 * 64 * 60
    # ... and these gain
    assert n(shape(16, 1, 8192, 16, 4, 64, 128)) == 2 * 16 * 16 * 2 * 129 * 4
    assert n(shape(1, 128, 8192, 4, 4, 64, 128)) == 32 * 128 * 4 * 2 * 129 * 4
    assert m(shape(1, 3000, 200, 2, 1, 32, 64)) == 94 * 64 * 60 + 2 * 11 * 128 * 128 * 4
    assert m(shape(2, 4001, 4001, 8, 2, 64, 128, causal=True)) == 4 * 252 * 64 * 60 + 128 * 4 * 128 * 256 * 4
