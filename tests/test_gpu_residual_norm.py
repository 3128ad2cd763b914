"""rib_residual_norm, its backward and rib_dropout against the fp64 oracle.

Tolerances, derived: outputs of a type with rounding unit eps/2 are off by at
most eps/2 of the value (half a step), plus the fp32 arithmetic before it. A
row's statistics are fp32 sums of C terms and a handful of products; K = 64
units of 2^-24 of the row's largest magnitudes (values, statistics times
weights) covers the chains here (a lane adds at most 8-12 terms, then 9
levels of a tree, twice, and about 20 products). Column sums add T terms in
chains of at most `chain` additions, each off by 2^-24 of the running sum,
which is at most the sum of magnitudes, plus K units for each term."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

EPS = 1e-5
K = 64 * 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _near(got, ref, dtype, slack, what):
    g = _np(got).reshape(ref.shape)
    assert np.all(np.isfinite(g)), f"{what}: not finite"
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + slack
    over = np.abs(g - ref) - tol
    assert over.max(initial=-1.0) <= 0, f"{what}: {np.abs(g - ref).max():.3e} off, {over.max():.3e} over"


def _make(T, C, xt, t, pre, post, gated, groups, seed=0, biases=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = {"x": n(T, C).to(xt), "y": (1.5 * n(T, C) + 0.2).to(t), "gate": torch.sigmoid(n(T, C)).to(t) if gated else None,
         "scale": 0.5 + 0.1 * n(groups, C) if groups else None}
    for k, kind in (("post", post), ("pre", pre)):
        a[k + "_w"] = 1 + 0.1 * n(C) if kind != "none" else None
        a[k + "_b"] = 0.1 * n(C) if kind == "layer" and biases else None
    a["dx_out"], a["dh"] = n(T, C).to(xt), n(T, C).to(t) if pre != "none" else None
    return a


ORDER = ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")


def _run(rib, a, T, C, xt, t, pre, post, rpg, p, seed=11, offset=5, step=None):
    d = {k: None if v is None else v.cuda() for k, v in a.items()}
    desc = rib.residual_norm_desc(T, C, xt, t, pre=pre, post=post, eps=EPS, rows_per_group=rpg, p=p, seed=seed, offset=offset)
    nan = lambda like: torch.full_like(like, float("nan"))  # noqa: E731
    x_out, h = nan(d["x"]), nan(d["y"]) if pre != "none" else None
    rib.rib_residual_norm(desc, d["x"], d["y"], *(d[k] for k in ORDER), x_out, h, step=step)
    out = {"x_out": x_out, "h": h}
    ws = torch.empty(rib.rib_residual_norm_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    grads = {"d" + k: nan(d[k]) if d[k] is not None else None for k in ("x", "y") + ORDER}
    rib.rib_residual_norm_bwd(desc, x_out, d["y"], *(d[k] for k in ORDER[:5]), d["dx_out"], d["dh"],
                              *(grads["d" + k] for k in ("x", "y") + ORDER), ws, step=step)
    out.update(grads)
    torch.cuda.synchronize()
    return out


def _check(rib, T, C, xt, t, pre, post, gated, groups, p, rpg=None, **kw):
    a = _make(T, C, xt, t, pre, post, gated, groups)
    rpg = rpg or max(1, -(-T // max(1, groups)))
    got = _run(rib, a, T, C, xt, t, pre, post, rpg, p, **kw)
    r = {k: _np(v) for k, v in a.items()}
    mask = bo.dropout_factor(T * C, p, 11, 5).reshape(T, C) if p else None
    o = dict(pre=pre, post=post, eps=EPS, rows_per_group=rpg, mask=mask)
    x1, h = bo.residual_norm(r["x"], r["y"], *(r[k] for k in ORDER), **o)
    # magnitudes that the fp32 slack scales with: what is added to form x'
    up = 1 / (1 - p)
    mag = np.abs(r["x"]).max() + up * 8 * (1 if r["scale"] is None else np.abs(r["scale"]).max())
    _near(got["x_out"], x1, xt, K * mag, "x_out")
    if pre != "none":
        # an error e of x' is at most 2 e r at h, r = 1/sqrt(var + eps) <= 316; here rows have unit spread
        rr = 1 / np.sqrt(((x1 - (x1.mean(1, keepdims=True) if pre == "layer" else 0)) ** 2).mean(1) + EPS)
        _near(got["h"], h, t, K * (mag * rr.max() + 8) * 1.5, "h")
    # the backward starts from the stored x_out
    g = bo.residual_norm_bwd(_np(got["x_out"]), r["y"], *(r[k] for k in ORDER[:5]), r["dx_out"], r["dh"], **o)
    ry = 1.0
    if post != "none":
        ry = (1 / np.sqrt(((r["y"] - (r["y"].mean(1, keepdims=True) if post == "layer" else 0)) ** 2).mean(1) + EPS)).max()
    rx = rr.max() if pre != "none" else 1.0
    big = (np.abs(g["dx"]).max() + 8 * rx) * 8
    _near(got["dx"], g["dx"], xt, K * big, "dx")
    _near(got["dy"], g["dy"], t, K * big * up * max(1.0, ry) * 8, "dy")
    if gated:
        _near(got["dgate"], g["dgate"], t, K * big * up * 8, "dgate")
    chain = (T + 7) // 8 + 512     # rows of a thread at most, then CTAs and slots
    for k in ORDER[1:]:
        if got["d" + k] is not None:
            _near(got["d" + k], g["d" + k], F32, (chain * 2.0 ** -24 + K * 8) * g[f"d{k}_abs"] + K * big * 1e-3, "d" + k)


SHAPES = [(1, 1), (4, 1), (17, 3), (300, 33), (65, 510), (31, 511), (12, 2045), (10, 2047), (9, 3001), (3, 2), (5, 7), (2, 8), (33, 48), (64, 180), (257, 180), (19, 255), (130, 256), (40, 1021), (21, 1024), (9, 2050),
          (6, 4095), (7, 4096)]


@pytest.mark.parametrize("T,C", SHAPES, ids=[f"{t}x{c}" for t, c in SHAPES])
def test_f32_stream_bf16_branch(cuda_lib, T, C):
    _check(cuda_lib, T, C, F32, BF16, "layer", "layer", True, 1, 0.0)


@pytest.mark.parametrize("pre,post", [("layer", "none"), ("rms", "layer"), ("none", "rms"), ("rms", "rms"), ("none", "none")])
@pytest.mark.parametrize("xt,t", [(F32, F32), (F32, F16), (BF16, BF16), (F16, F16)])
def test_norm_kinds_and_types(cuda_lib, pre, post, xt, t):
    _check(cuda_lib, 50, 180, xt, t, pre, post, True, 1, 0.1)


@pytest.mark.parametrize("T,rpg", [(48, 16), (50, 16), (7, 1), (700, 233)])
def test_scale_of_row_groups(cuda_lib, T, rpg):
    _check(cuda_lib, T, 52, F32, BF16, "layer", "rms", False, -(-T // rpg), 0.0, rpg=rpg)


@pytest.mark.parametrize("C", [180, 37, 2048])
def test_dropout_inside_the_join(cuda_lib, C):
    _check(cuda_lib, 61, C, F32, BF16, "rms", "layer", True, 1, 0.35)


def test_many_rows_same_bits_twice(cuda_lib):
    T, C = 20000, 180
    a = _make(T, C, F32, BF16, "layer", "layer", True, 1)
    one = _run(cuda_lib, a, T, C, F32, BF16, "layer", "layer", T, 0.1)
    two = _run(cuda_lib, a, T, C, F32, BF16, "layer", "layer", T, 0.1)
    for k in one:
        assert torch.equal(one[k], two[k]), k
    _check(cuda_lib, T, C, F32, BF16, "layer", "layer", True, 1, 0.1)


def test_unaligned_rows_take_the_scalar_form(cuda_lib):
    """The same values through a buffer shifted by one element."""
    rib, T, C = cuda_lib, 33, 180
    a = _make(T, C, F32, BF16, "layer", "none", False, 0)
    desc = rib.residual_norm_desc(T, C, F32, BF16, pre="layer", post="none", eps=EPS)
    x, y = a["x"].cuda(), a["y"].cuda()
    ref_x, ref_h = torch.empty_like(x), torch.empty_like(y)
    rib.rib_residual_norm(desc, x, y, x_out=ref_x, h=ref_h)
    buf = torch.full((T * C + 2,), float("nan"), dtype=BF16, device="cuda")
    ys = buf[1:1 + T * C]
    ys.copy_(y.view(-1))
    h = torch.empty_like(y)
    x_out = torch.empty_like(x)
    rib.rib_residual_norm(desc, x, ys, x_out=x_out, h=h)
    assert torch.equal(ref_x, x_out)       # elementwise: the same products and sums
    assert (h.float() - ref_h.float()).abs().max() <= 2 ** -7 * ref_h.float().abs().max()   # a row sum's order differs
    assert torch.isnan(buf[0]) and torch.isnan(buf[-1])


def test_pre_norm_alone_and_in_place(cuda_lib):
    rib, T, C = cuda_lib, 65, 48
    a = _make(T, C, F32, BF16, "layer", "none", False, 0)
    x, w, b = a["x"].cuda(), a["pre_w"].cuda(), a["pre_b"].cuda()
    desc = rib.residual_norm_desc(T, C, F32, BF16, pre="layer")
    h = torch.empty(T, C, dtype=BF16, device="cuda")
    rib.rib_residual_norm(desc, x, pre_w=w, pre_b=b, h=h)
    ref = torch.empty_like(h)
    rib.rib_layernorm(x, ref, T, C, w, b, EPS)
    assert (h.float() - ref.float()).abs().max() <= 2 ** -7 * ref.float().abs().max()
    _, r = bo.residual_norm(_np(x), pre_w=_np(w), pre_b=_np(b))
    _near(h, r, BF16, K * 32, "h")
    dh = a["dh"].cuda()
    dx, ws = torch.empty_like(x), torch.empty(rib.rib_residual_norm_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(b)
    rib.rib_residual_norm_bwd(desc, x, pre_w=w, dh=dh, dx=dx, dpre_w=dw, dpre_b=db, workspace=ws)
    g = bo.residual_norm_bwd(_np(x), pre_w=_np(w), dh=_np(dh))
    _near(dx, g["dx"], F32, K * 64, "dx")
    _near(dw, g["dpre_w"], F32, K * 8 * g["dpre_w_abs"] + 1e-7, "dpre_w")
    # in place: the stream over x, h over y, dx over dx_out, dy over dh
    y = a["y"].cuda()
    x1, h1 = torch.empty_like(x), torch.empty_like(y)
    rib.rib_residual_norm(desc, x, y, pre_w=w, pre_b=b, x_out=x1, h=h1)
    xi, yi = x.clone(), y.clone()
    rib.rib_residual_norm(desc, xi, yi, pre_w=w, pre_b=b, x_out=xi, h=yi)
    assert torch.equal(xi, x1) and torch.equal(yi, h1)
    dxo = a["dx_out"].cuda()
    dx1, dy1 = torch.empty_like(x), torch.empty_like(y)
    rib.rib_residual_norm_bwd(desc, x1, y, pre_w=w, dx_out=dxo, dh=dh, dx=dx1, dy=dy1)
    dxi, dhi = dxo.clone(), dh.clone()
    rib.rib_residual_norm_bwd(desc, x1, y, pre_w=w, dx_out=dxi, dh=dhi, dx=dxi, dy=dhi)
    assert torch.equal(dxi, dx1) and torch.equal(dhi, dy1)


def test_no_rows(cuda_lib):
    rib, C = cuda_lib, 48
    desc = rib.residual_norm_desc(0, C, F32, BF16, pre="layer", post="layer")
    e = lambda t: torch.empty(0, C, dtype=t, device="cuda")  # noqa: E731
    w = torch.ones(C, device="cuda")
    rib.rib_residual_norm(desc, e(F32), e(BF16), post_w=w, pre_w=w, x_out=e(F32), h=e(BF16))
    assert rib.rib_residual_norm_bwd_workspace_size(desc) == 0
    dw = [torch.full((C,), float("nan"), device="cuda") for _ in range(4)]
    rib.rib_residual_norm_bwd(desc, e(F32), e(BF16), None, None, w, w, w, e(F32), e(BF16), e(F32), e(BF16), None, None, *dw,
                              workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert all(bool((d == 0).all()) for d in dw)


def test_constant_and_huge_rows(cuda_lib):
    """A constant row has LayerNorm 0 and a finite gradient; offsets of 1e4 lose no more than fp32 holds."""
    rib, T, C = cuda_lib, 4, 180
    desc = rib.residual_norm_desc(T, C, F32, F32, pre="layer")
    x = torch.zeros(T, C)
    x[1] = 3.0
    x[2] = 1e4 + torch.randn(C, generator=torch.Generator().manual_seed(0))
    x[3] = torch.randn(C, generator=torch.Generator().manual_seed(1)) * 1e15
    xc, h = x.cuda(), torch.empty(T, C, device="cuda")
    rib.rib_residual_norm(desc, xc, h=h)
    _, r = bo.residual_norm(_np(xc))
    assert torch.all(h[0] == 0)
    assert h[1].abs().max() <= 3 * 2.0 ** -20 / EPS ** 0.5    # the mean of equal values, rounded, over sqrt(eps)
    assert np.abs(_np(h[2]) - r[2]).max() <= 1e4 * 2.0 ** -20   # values of 1e4 are 2^-24 of themselves exact, deviations of 1
    assert np.abs(_np(h[3]) - r[3]).max() <= K * 8


def test_masked_branch_values_do_not_leak(cuda_lib):
    """Infinities and NaN in dropped elements of the branch leave the stream as it was."""
    rib, T, C, p = cuda_lib, 20, 64, 0.5
    a = _make(T, C, F32, BF16, "none", "none", False, 0)
    f = torch.from_numpy(bo.dropout_factor(T * C, p, 11, 5)).view(T, C)
    y = a["y"].masked_fill(f == 0, float("nan"))
    y[0] = torch.where(f[0] == 0, float("inf"), y[0].double()).to(BF16)
    desc = rib.residual_norm_desc(T, C, F32, BF16, pre="none", p=p, seed=11, offset=5)
    out = torch.empty(T, C, device="cuda")
    rib.rib_residual_norm(desc, a["x"].cuda(), y.cuda(), x_out=out)
    ref = a["x"].double() + torch.where(f > 0, f * torch.nan_to_num(y.double()), 0.0)
    assert (out.cpu().double() - ref).abs().max() <= K * 16


# ------------------------------------------------------------------- dropout
@pytest.mark.parametrize("t", [BF16, F16, F32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 4095, 4096, 4097, 100_003])
def test_dropout_matches_the_oracle(cuda_lib, t, n):
    x = torch.randn(n, generator=torch.Generator().manual_seed(n)).to(t)
    seed, offset, p = 0xFEDCBA9876543210, (5 << 32) + 77, 0.3
    f = bo.dropout_factor(n, p, seed, offset)
    for shift in (0, 1):
        buf = torch.full((n + 3,), float("nan"), dtype=t, device="cuda")
        xs = torch.zeros(n + 1, dtype=t, device="cuda")[shift:shift + n]
        xs.copy_(x)
        cuda_lib.rib_dropout(xs, buf[shift:shift + n], p, seed, offset)
        got = buf[shift:shift + n]
        ref = _np(x) * f
        assert np.array_equal(_np(got) == 0, (f == 0) | (_np(x) == 0))
        _near(got, ref, t, 2.0 ** -23 * np.abs(ref) + (2.0 ** -25 if t == F16 else 0), "y")
        assert torch.isnan(buf[shift + n:]).all() and torch.isnan(buf[:shift]).all()


def test_dropout_edges_in_place_step_and_replay(cuda_lib):
    rib = cuda_lib
    x = torch.randn(5000, device="cuda")
    y = torch.empty_like(x)
    rib.rib_dropout(x, y, 0.0, 3)
    assert torch.equal(x, y)
    rib.rib_dropout(torch.full_like(x, float("inf")), y, 1.0, 3)
    assert torch.all(y == 0)
    rib.rib_dropout(x, y, 0.4, 3, 12)
    z = x.clone()
    rib.rib_dropout(z, z, 0.4, 3, 12)
    assert torch.equal(y, z)
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    rib.rib_dropout(x, z, 0.4, 3, 7, step=step)
    assert torch.equal(y, z)
    # a captured call draws the mask of the step that the program sets before each replay
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rib.rib_dropout(x, z, 0.4, 3, 7, step=step)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rib.rib_dropout(x, z, 0.4, 3, 7, step=step)
    for s in (5, 6, 5):
        step.fill_(s)
        graph.replay()
        rib.rib_dropout(x, y, 0.4, 3, 7 + s)
        assert torch.equal(y, z), s
    rib.rib_dropout(torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), 0.5, 1)


def test_step_reaches_the_join(cuda_lib):
    T, C = 30, 60
    a = _make(T, C, F32, BF16, "layer", "layer", True, 1)
    step = torch.tensor([3], dtype=torch.int64, device="cuda")
    one = _run(cuda_lib, a, T, C, F32, BF16, "layer", "layer", T, 0.2, offset=5)
    two = _run(cuda_lib, a, T, C, F32, BF16, "layer", "layer", T, 0.2, offset=2, step=step)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_two_host_threads(cuda_lib):
    """Host threads run joins of two widths of one kernel instance, whose shared memory differs, on their own streams:
    every call is accepted, and its results are those of a call alone."""
    rib, T = cuda_lib, 2
    lib, jobs = rib.load(), []
    for C in (2048, 4092, 2048, 4092):
        g = torch.Generator().manual_seed(C)
        x, y, gate = torch.randn(T, C, generator=g).cuda(), *(torch.randn(T, C, generator=g).to(BF16).cuda() for _ in range(2))
        desc = rib.residual_norm_desc(T, C, F32, BF16, pre="layer", post="layer", eps=EPS)
        alone, out = ([torch.empty_like(t) for t in (x, y, x, y)] for _ in range(2))
        rib.rib_residual_norm(desc, x, y, gate, x_out=alone[0], h=alone[1])
        rib.rib_residual_norm_bwd(desc, alone[0], y, gate, dx_out=x, dh=y, dx=alone[2], dy=alone[3])
        jobs.append((desc, x, y, gate, alone, out, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(desc, x, y, gate, alone, out, stream, failed):
        # arguments made once: most of a thread's time is spent inside the library, without the interpreter's lock
        p, c = (lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())), ctypes.byref(desc)
        st, x1 = ctypes.c_void_p(stream.cuda_stream), out[0]
        fwd = [p(t) for t in (x, y, gate, None, None, None, None, None, x1, out[1], None)]
        bwd = [p(t) for t in (x1, y, gate, None, None, None, None, x, y, out[2], out[3], *[None] * 6)]
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(8000):
            if lib.rib_residual_norm(c, *fwd, st) or lib.rib_residual_norm_bwd(c, *bwd, None, 0, None, st):
                failed.append(lib.rib_last_error().decode())
                return

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    rib.rib_device_error()
    for desc, _, _, _, alone, out, _, failed in jobs:
        assert not failed, failed
        for a, b in zip(alone, out):
            assert torch.equal(a, b), desc.C


@pytest.mark.parametrize("C", [64, 37, 2050])
@pytest.mark.parametrize("post", ["none", "layer"])
def test_dropped_elements_have_no_gradient(cuda_lib, C, post):
    """Infinities and NaN in the branch (without a post norm), the gate and the scale of dropped elements change nothing, to
    the bit; the gradients are the oracle's."""
    T, p = 24, 0.5
    a = _make(T, C, F32, BF16, "layer", post, True, T)
    dropped = torch.from_numpy(bo.dropout_factor(T * C, p, 11, 5) == 0).view(T, C)
    bad = {k: v if v is None else v.clone() for k, v in a.items()}
    for i, k in enumerate(("gate", "scale") + (("y",) if post == "none" else ())):
        for j, v in enumerate((float("nan"), float("inf"), -float("inf"))):
            bad[k][dropped & ((torch.arange(T) + i)[:, None] % 3 == j)] = v
    args = (T, C, F32, BF16, "layer", post, 1, p)
    want, got = _run(cuda_lib, a, *args), _run(cuda_lib, bad, *args)
    for k, v in want.items():
        if v is not None:
            assert torch.isfinite(v).all(), k
            assert torch.equal(v, got[k]), f"{k}: {int((v != got[k]).sum())} of {v.numel()} differ"
    _check(cuda_lib, T, C, F32, BF16, "layer", post, True, T, p, rpg=1)


@pytest.mark.parametrize("groups", [1, 3])
def test_weights_of_a_flat_buffer(cuda_lib, groups):
    """Weights are read one element at a time: slices of a parameter buffer that start off a 16-byte boundary give the bits of
    aligned ones (the same vectors and the same order of sums), and their gradients go into such slices."""
    rib, T, C, p = cuda_lib, 51, 180, 0.1
    a = _make(T, C, F32, BF16, "layer", "layer", True, groups)
    rpg = T // groups
    want = _run(rib, a, T, C, F32, BF16, "layer", "layer", rpg, p)
    names = ORDER[1:]
    at, n = {}, 1
    for k in names:
        at[k] = (n, n + a[k].numel())
        n += a[k].numel() + 1
    flat, grads = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    w, dw = ({k: b[at[k][0]:at[k][1]].view(a[k].shape) for k in names} for b in (flat, grads))
    d = {k: v.cuda() for k, v in a.items()}
    for k in names:
        w[k].copy_(a[k])
    assert any(w[k].data_ptr() % 16 for k in names)
    desc = rib.residual_norm_desc(T, C, F32, BF16, pre="layer", post="layer", eps=EPS, rows_per_group=rpg, p=p, seed=11, offset=5)
    x_out, h, dx, dy, dgate = (torch.empty_like(d[k]) for k in ("x", "y", "x", "y", "gate"))
    rib.rib_residual_norm(desc, d["x"], d["y"], d["gate"], *(w[k] for k in names), x_out, h)
    ws = torch.empty(rib.rib_residual_norm_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    rib.rib_residual_norm_bwd(desc, x_out, d["y"], d["gate"], *(w[k] for k in names[:4]), d["dx_out"], d["dh"], dx, dy, dgate,
                              *(dw[k] for k in names), ws)
    got = {"x_out": x_out, "h": h, "dx": dx, "dy": dy, "dgate": dgate, **{"d" + k: dw[k] for k in names}}
    for k, v in got.items():
        assert torch.equal(v, want[k]), k
    assert int(torch.isnan(grads).sum()) == n - sum(a[k].numel() for k in names)     # nothing between the slices


def test_tensors_of_other_shapes_are_refused(cuda_lib):
    """Tensors hold the descriptor's rows of C values: flat or any shape that ends in C, no more and no fewer."""
    rib, T, C = cuda_lib, 6, 40
    f = lambda *s, t=F32: torch.randn(*s, device="cuda").to(t)  # noqa: E731
    desc = rib.residual_norm_desc(T, C, F32, BF16, pre="layer", post="layer", rows_per_group=3)
    ok = {"x": f(T, C), "y": f(T, C, t=BF16), "gate": f(T, C, t=BF16), "scale": f(2, C), "post_w": f(C), "post_b": f(C), "pre_w": f(C),
          "pre_b": f(C), "x_out": f(T, C), "h": f(T, C, t=BF16)}
    rib.rib_residual_norm(desc, **ok)
    for k, v in ok.items():
        for bad in (f(2 * v.numel() // C, C), f(C, v.numel() // C), f(v.numel() - C), f(v.numel() + C)):
            with pytest.raises(ValueError, match=k):
                rib.rib_residual_norm(desc, **{**ok, k: bad.to(v.dtype)})
    for shape in ((T * C,), (2, 3, C), (1, T, 1, C)):
        out = {k: torch.empty(shape, device="cuda", dtype=ok[k].dtype) for k in ("x_out", "h")}
        rib.rib_residual_norm(desc, **{**ok, **{k: ok[k].view(shape) for k in ("x", "y", "gate")}, **out})
        assert all(torch.equal(out[k].view(T, C), ok[k]) for k in out)
    grads = {"d" + k: torch.empty_like(ok[k]) for k in ("x", "y", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b")}
    args = {k: ok[k] for k in ("x_out", "y", "gate", "scale", "post_w", "post_b", "pre_w")}
    args.update(grads, dx_out=f(T, C), dh=f(T, C, t=BF16),
                workspace=torch.empty(rib.rib_residual_norm_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda"))
    rib.rib_residual_norm_bwd(desc, **args)
    for k, v in args.items():
        if k != "workspace":
            with pytest.raises(ValueError, match=k):
                rib.rib_residual_norm_bwd(desc, **{**args, k: torch.empty(C, v.numel() // C, device="cuda", dtype=v.dtype)})
    # no rows: a scale of any number of rows
    none = rib.residual_norm_desc(0, C, F32, BF16, pre="layer")
    e = lambda t: torch.empty(0, C, dtype=t, device="cuda")  # noqa: E731
    rib.rib_residual_norm(none, e(F32), e(BF16), scale=f(1, C), x_out=e(F32), h=e(BF16))
    rib.rib_residual_norm_bwd(none, e(F32), e(BF16), scale=f(1, C), dx_out=e(F32), dh=e(BF16), dscale=f(1, C), dx=e(F32), dy=e(BF16))
    rib.rib_residual_norm_bwd(none, e(F32), e(BF16), dx_out=e(F32), dh=e(BF16), dscale=f(1, C), dx=e(F32), dy=e(BF16))


@pytest.mark.parametrize("T,rpg,C", [(50, 17, 37), (9, 1, 51), (31, 5, 1021), (8, 3, 2047), (60, 7, 3), (45, 11, 46)])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_row_groups_at_odd_widths(cuda_lib, T, rpg, C, p):
    """Groups that start on odd rows, whose rows of an odd width start one element early in pairs."""
    _check(cuda_lib, T, C, F32, BF16, "rms", "layer", True, -(-T // rpg), p, rpg=rpg)


@pytest.mark.parametrize("C", [8, 37, 180, 1021])
@pytest.mark.parametrize("xt,t", [(F32, BF16), (F16, F16)])
def test_tensors_off_a_16_byte_boundary(cuda_lib, C, xt, t, monkeypatch):
    """Every [T, C] tensor starts one element into its buffer, forward and backward: the oracle's values, and nothing around
    the tensors is written."""
    rib, buffers = cuda_lib, []

    def shifted(v):
        if v is None or v.dim() != 2 or v.shape[0] != T:
            return v
        buf = torch.full((v.numel() + 9,), 7.0, dtype=v.dtype, device="cuda")
        w = buf[1:1 + v.numel()].view(v.shape)
        w.copy_(v)
        buffers.append((buf, v.numel()))
        return w

    T = 37
    run = {n: getattr(rib, n) for n in ("rib_residual_norm", "rib_residual_norm_bwd")}

    def through(name):
        def call(desc, *args, step=None):
            own = [shifted(a) if torch.is_tensor(a) else a for a in args]
            run[name](desc, *own, step=step)
            for a, b in zip(args, own):
                if a is not b:
                    a.copy_(b)
        return call

    for n in run:
        monkeypatch.setattr(rib, n, through(n))
    _check(rib, T, C, xt, t, "layer", "layer", True, 1, 0.2)
    assert len(buffers) == 5 + 8      # x, y, gate, x_out, h; x_out, y, gate, dx_out, dh, dx, dy, dgate
    for buf, n in buffers:
        assert buf[0] == 7 and bool((buf[1 + n:] == 7).all())
