"""rib_diff_attention and its backward against a dense fp64 form of the
definition on the same rounded inputs.

Tolerances, derived; u is half a step of the 16-bit type.
* Probabilities take the type for the products: u of each, so a sum of a_j v_j
  is off by u sum a_j |v_j|; a result is rounded once more, u of itself.
* K bounds the relative error of a probability before that: the fp32 score has
  d products and sums, each off by 2^-24 of scale sum |q k| at most, the
  exponent's argument and the row's sum a few more.
* fp16 probabilities below its smallest normal value are off by half of its
  smallest step, 2^-25 (the largest of a row is at least 1 in the forward; the
  backward holds them times 64: 2^-31).
* D_i = dO . O_i inherits the errors of o and o2 (the bounds above), and the
  fp32 sum's.
Worst-case sums are far above what independent roundings leave, so where a
tensor has enough values the root mean square of its error is bounded too: the
roundings of P, of dS, of D and of the result each add at most u / sqrt(3) of
sums as large as the result; 4 u covers them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("q1", "q2", "k1", "k2", "v")


def _inputs(B, Nq, Nk, Hq, Hk, d, dv, t, seed=0, lam_t=None):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    x = {"q1": n(B, Nq, Hq, d), "q2": n(B, Nq, Hq, d), "k1": n(B, Nk, Hk, d), "k2": n(B, Nk, Hk, d), "v": n(B, Nk, Hk, dv)}
    x["lam"] = (torch.rand(Hq, generator=g) * 1.6 - 0.6).to(lam_t or t).cuda()
    x["do"] = n(B, Nq, Hq, dv)
    return x


def _seqs(x, lens, causal, window, width):
    B, Nq, Nk = x["q1"].shape[0], x["q1"].shape[1], x["k1"].shape[1]
    for b in range(B):
        if window:
            H = Nq // width
            at = torch.arange(Nq).reshape(H, width)
            for y in range(0, H, window):
                for c in range(0, width, window):
                    r = at[y:y + window, c:c + window].reshape(-1).cuda()
                    yield b, r, r, None
        else:
            n = Nk if lens is None else min(max(int(lens[b]), 0), Nk)
            hide = None
            if causal:
                hide = torch.arange(n, device="cuda")[None] > torch.arange(Nq, device="cuda")[:, None] + n - Nq
            yield b, torch.arange(Nq, device="cuda"), torch.arange(n, device="cuda"), hide


def _reference(x, scale, t, lens=None, causal=False, window=0, width=0):
    """Values and tolerances by name."""
    u, half = torch.finfo(t).eps / 2, t == F16
    f = {k: v.double() for k, v in x.items()}
    B, Nq, Hq, d = x["q1"].shape
    G = Hq // x["k1"].shape[2]
    val = {"o": torch.zeros_like(f["do"]), "o2": torch.zeros_like(f["do"]), "lse": torch.full((2, B, Hq, Nq), -math.inf, device="cuda").double()}
    val.update({"d" + k: torch.zeros_like(f[k]) for k in NAMES})
    val["dlam"] = torch.zeros(Hq, device="cuda").double()
    tol = {k: torch.zeros_like(v) for k, v in val.items()}
    for b, qr, kr, hide in _seqs(x, lens, causal, window, width):
        for h in range(Hq if len(kr) else 0):
            g = h // G
            q1, q2, k1, k2, v = (f[n][b, r, hh] for n, r, hh in (("q1", qr, h), ("q2", qr, h), ("k1", kr, g), ("k2", kr, g), ("v", kr, g)))
            do, lam = f["do"][b, qr, h], f["lam"][h]
            al, n = lam.abs(), len(kr)
            big = max((q1.abs() @ k1.abs().T).max().item(), (q2.abs() @ k2.abs().T).max().item()) * scale
            K = ((d + 8) * (big + 4) + n / 4 + 64) * 2.0 ** -24
            low, low_b = (n * 2.0 ** -25, 2.0 ** -31) if half else (0.0, 0.0)
            a = []
            for i, (q, k) in enumerate(((q1, k1), (q2, k2))):
                s = q @ k.T * scale
                if hide is not None:
                    s = s.masked_fill(hide, -math.inf)
                m = s.amax(1, keepdim=True)
                m = torch.where(m > -math.inf, m, 0.0)
                p = torch.exp(s - m)
                l = p.sum(1, keepdim=True)
                a.append(p / torch.where(l > 0, l, 1.0))
                lse = (m + torch.log(l))[:, 0]
                val["lse"][i, b, h, qr] = lse
                tol["lse"][i, b, h, qr] = torch.where(lse > -math.inf, K + lse.abs() * 2.0 ** -22, 0.0)
            va = v.abs()
            s1, s2 = a[0] @ va, a[1] @ va
            o2 = a[1] @ v
            o = a[0] @ v - lam * o2
            vm = va.max()
            t2 = u * o2.abs() + (u + K) * s2 + low * vm
            to = u * o.abs() + (u + K) * (s1 + al * s2) + (1 + al) * low * vm
            val["o"][b, qr, h], val["o2"][b, qr, h], tol["o"][b, qr, h], tol["o2"][b, qr, h] = o, o2, to, t2
            da, dp = do.abs(), do @ v.T
            e32 = 2.0 ** -24 * (v.shape[1] + 8)
            dpe = e32 * (da @ va.T)                         # fp32 sums of dP
            d2 = (do * o2).sum(1, keepdim=True)
            d1 = (do * (o + lam * o2)).sum(1, keepdim=True)
            e2 = (da * (t2 + e32 * o2.abs())).sum(1, keepdim=True)
            e1 = (da * (to + al * t2 + e32 * (o.abs() + al * o2.abs()))).sum(1, keepdim=True)
            val["dlam"][h] -= d2.sum()
            tol["dlam"][h] += e2.sum() + 2.0 ** -24 * 64 * d2.abs().sum()
            val["dv"][b, kr, g] += (a[0] - lam * a[1]).T @ do
            tol["dv"][b, kr, g] += (u + 2 * K) * ((a[0] + al * a[1]).T @ da) + len(qr) * low_b * da.max()
            for ai, q, k, dn, en, nq, nk, c in ((a[0], q1, k1, d1, e1, "dq1", "dk1", 1.0), (a[1], q2, k2, d2, e2, "dq2", "dk2", -lam)):
                ds = c * ai * (dp - dn)
                es = (u + 4 * K) * ds.abs() + abs(c) * ai * (dpe + en + 2.0 ** -22 * (dp.abs() + dn.abs())) + low_b
                if hide is not None:
                    es = es.masked_fill(hide, 0.0)
                val[nq][b, qr, h] = scale * (ds @ k)
                tol[nq][b, qr, h] = scale * (es @ k.abs())
                val[nk][b, kr, g] += scale * (ds.T @ q)
                tol[nk][b, kr, g] += scale * (es.T @ q.abs())
    for k in ("dq1", "dq2", "dk1", "dk2", "dv"):
        tol[k] += u * val[k].abs() + (2.0 ** -25 if half else 0.0)
    tol["dlam"] += torch.finfo(x["lam"].dtype).eps / 2 * val["dlam"].abs()
    return val, tol


def _run(rib, x, scale, t, lens=None, causal=False, window=0, width=0, train=True, strides=None, layout=lambda k, v: v):
    """Outputs by name, started from NaN."""
    B, Nq, Hq, d = x["q1"].shape
    Nk, Hk, dv = x["v"].shape[1:]
    desc = rib.diff_attn_desc(B, Nq, Nk, Hq, Hk, d, dv, scale, t, lam_dtype=x["lam"].dtype, causal=causal, window=window, width=width,
                              **(strides or {}))
    nan = lambda k, v: layout(k, torch.full_like(v, float("nan")))  # noqa: E731
    x = {k: layout(k, v) for k, v in x.items()}
    ws = lambda n: torch.full((n // 4,), float("nan"), device="cuda")  # noqa: E731
    out = {"o": nan("do", x["do"])}
    if train:
        out["o2"], out["lse"] = nan("do", x["do"]), torch.full((2, B, Hq, Nq), float("nan"), device="cuda")
    args = [x[k] for k in NAMES + ("lam",)] + [lens]
    rib.rib_diff_attention(desc, *args, out["o"], out.get("o2"), out.get("lse"), ws(rib.rib_diff_attention_workspace_size(desc)))
    if train:
        grads = {"d" + k: nan(k, x[k]) for k in NAMES}
        grads["dlam"] = torch.full_like(x["lam"], float("nan"))
        rib.rib_diff_attention_bwd(desc, *args, out["o"], out["o2"], out["lse"], x["do"], *grads.values(),
                                   ws(rib.rib_diff_attention_bwd_workspace_size(desc)))
        out.update(grads)
    torch.cuda.synchronize()
    rib.rib_device_error()
    return out


def _compare(got, val, tol, t, rms=()):
    for k, g in got.items():
        g, r = g.double(), val[k]
        same = (g == r) & torch.isinf(r)          # the log-sum-exp of rows that see nothing
        off = torch.where(same, 0.0, (g - r).abs() - tol[k])
        assert not torch.isnan(off).any(), f"{k}: {int(torch.isnan(off).sum())} of {off.numel()} not finite"
        if off.numel():
            assert off.max() <= 0, f"{k}: {float((g - r).abs()[~same].max()):.3e} off, {float(off.max()):.3e} over"
        if k in rms:
            e = float((g - r).square().mean().sqrt() / r.square().mean().sqrt())
            assert e <= 4 * torch.finfo(t).eps / 2, f"{k}: root mean square error {e:.2e}"


def _check(rib, B, Nq, Nk, Hq, Hk, d, dv, t, lens=None, train=True, rms=(), lam_t=None, seed=0, **kw):
    x = _inputs(B, Nq, Nk, Hq, Hk, d, dv, t, seed, lam_t)
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = d ** -0.5
    got = _run(rib, x, scale, t, lens, train=train, **kw)
    val, tol = _reference(x, scale, t, lens, **kw)
    _compare(got, val, tol, t, rms)


ALL = ("o", "o2", "dq1", "dq2", "dk1", "dk2", "dv")
WIDTHS = [(16, 32), (8, 8), (32, 64), (24, 40), (24, 64), (32, 40), (16, 64), (64, 128), (64, 64), (40, 16), (48, 104)]


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("d,dv", WIDTHS, ids=[f"{a}-{b}" for a, b in WIDTHS])
def test_widths_and_types(cuda_lib, d, dv, t):
    _check(cuda_lib, 2, 150, 190, 2, 2, d, dv, t, rms=ALL)


@pytest.mark.parametrize("n", [1, 2, 15, 63, 64, 65, 127, 128, 129, 257, 1000])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(cuda_lib, n, causal):
    _check(cuda_lib, 1, n, n, 2, 1, 32, 64, BF16, causal=causal)


@pytest.mark.parametrize("Nq,Nk", [(1, 300), (5, 130), (200, 70), (130, 1), (300, 129)])
@pytest.mark.parametrize("causal", [False, True])
def test_different_lengths(cuda_lib, Nq, Nk, causal):
    """Causal with more queries than keys: the first rows see nothing."""
    _check(cuda_lib, 2, Nq, Nk, 3, 3, 16, 32, F16, causal=causal)


@pytest.mark.parametrize("Hq,Hk", [(8, 1), (6, 2), (5, 5), (24, 8), (7, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_key_heads(cuda_lib, Hq, Hk, causal):
    _check(cuda_lib, 2, 77, 77, Hq, Hk, 64, 128, BF16, causal=causal, rms=ALL)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dv", [(16, 32), (64, 128)])
def test_key_lengths(cuda_lib, causal, d, dv):
    """Lengths of zero, one, inside a tile, on its edge, full, and beyond the tensors."""
    _check(cuda_lib, 8, 70, 260, 2, 1, d, dv, BF16, lens=[0, 1, 64, 127, 128, 200, 260, 1000], causal=causal)
    _check(cuda_lib, 2, 70, 260, 2, 1, d, dv, BF16, lens=[-3, 0], causal=causal)


@pytest.mark.parametrize("H,W,window", [(8, 8, 8), (32, 32, 16), (7, 5, 8), (13, 29, 8), (31, 31, 12), (9, 40, 31), (40, 33, 32), (3, 1, 2),
                                        (1, 17, 4), (65, 70, 64), (16, 16, 1)])
def test_windows(cuda_lib, H, W, window):
    _check(cuda_lib, 2, H * W, H * W, 3, 3, 16, 32, BF16, window=window, width=W)


def test_windows_with_shared_heads(cuda_lib):
    _check(cuda_lib, 1, 30 * 22, 30 * 22, 6, 2, 32, 64, F16, window=16, width=22, rms=ALL)


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("t", [BF16, F16])
def test_single_tokens_over_long_keys(cuda_lib, G, t):
    """Few rows: the keys are split and joined, parts without keys among them."""
    _check(cuda_lib, 5, 1, 4099, 2 * G, 2, 64, 128, t, lens=[4099, 1, 0, 2048, 130], rms=("o",))
    _check(cuda_lib, 1, 4, 9000, G, 1, 16, 32, t, causal=True, rms=("o",))


@pytest.mark.parametrize("Nq,G,Nk", [(6, 5, 3000), (32, 1, 2000), (3, 10, 5000), (2, 16, 1300), (33, 1, 4000)])
def test_few_rows_over_split_keys(cuda_lib, Nq, G, Nk):
    """Up to 32 rows a key head stand in every lane quarter; 33 do not. With the backward."""
    _check(cuda_lib, 1, Nq, Nk, G, 1, 32, 64, BF16, rms=("o", "o2", "dv"))
    _check(cuda_lib, 2, Nq, Nk, 2 * G, 2, 16, 32, F16, lens=[Nk - 77, 70], causal=True)


def test_many_heads_on_one_key_head(cuda_lib):
    _check(cuda_lib, 1, 70, 70, 64, 1, 16, 32, BF16, causal=True)
    _check(cuda_lib, 1, 90, 90, 33, 1, 32, 64, BF16)


@pytest.mark.parametrize("H,W,window", [(26, 29, 12), (20, 40, 31), (16, 16, 8)])
def test_a_bad_window_stays_in_its_window(cuda_lib, H, W, window):
    """NaN in every tensor of one window: the others' results are the same bits."""
    t, N = BF16, H * W
    x = _inputs(1, N, N, 2, 1, 16, 32, t)
    one = _run(cuda_lib, x, 0.25, t, window=window, width=W)
    bad = torch.zeros(H, W, dtype=torch.bool, device="cuda")
    bad[window:2 * window, :window] = True
    bad = bad.reshape(-1)
    for k in NAMES + ("do",):
        x[k][0, bad] = float("nan")
    two = _run(cuda_lib, x, 0.25, t, window=window, width=W)
    for k in ("o", "o2", "dq1", "dq2", "dk1", "dk2", "dv"):
        assert torch.equal(one[k][0, ~bad], two[k][0, ~bad]), k
        assert torch.isnan(two[k][0, bad]).all(), k
    assert torch.equal(one["lse"][..., ~bad], two["lse"][..., ~bad])


def test_two_calls_at_once(cuda_lib):
    """Two streams, each with its own outputs and workspace."""
    rib, t = cuda_lib, BF16
    xs = [_inputs(1, 700, 700, 4, 2, 32, 64, t, seed=s) for s in (1, 2)]
    want = [_run(rib, x, 0.2, t, causal=True) for x in xs]
    desc = rib.diff_attn_desc(1, 700, 700, 4, 2, 32, 64, 0.2, t, causal=True)
    streams, outs, keep = [torch.cuda.Stream() for _ in xs], [], []
    torch.cuda.synchronize()
    for x, st in zip(xs, streams):
        out = {k: torch.full_like(v, float("nan")) for k, v in want[0].items()}
        ws = torch.empty(max(1, rib.rib_diff_attention_workspace_size(desc)), dtype=torch.uint8, device="cuda")
        wb = torch.empty(rib.rib_diff_attention_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        outs.append(out)
        keep.append((ws, wb))
    for _ in range(3):
        for x, st, out, (ws, wb) in zip(xs, streams, outs, keep):
            args = [x[k] for k in NAMES + ("lam",)] + [None]
            rib.rib_diff_attention(desc, *args, out["o"], out["o2"], out["lse"], ws, stream=st)
            rib.rib_diff_attention_bwd(desc, *args, out["o"], out["o2"], out["lse"], x["do"], *(out["d" + k] for k in NAMES + ("lam",)), wb,
                                       stream=st)
    torch.cuda.synchronize()
    for w, out in zip(want, outs):
        for k in w:
            assert torch.equal(w[k], out[k]), k


def test_long_sequences(cuda_lib):
    _check(cuda_lib, 1, 4500, 4500, 2, 1, 64, 128, BF16, causal=True, rms=ALL)
    _check(cuda_lib, 1, 6000, 6000, 1, 1, 16, 32, F16, rms=ALL)


@pytest.mark.parametrize("t", [BF16, F16])
def test_split_key_sums(cuda_lib, t):
    """Few key tiles over many rows: their sums are split and added, empty shares and keys behind a length among them."""
    _check(cuda_lib, 1, 3000, 200, 2, 1, 32, 64, t, rms=ALL)
    _check(cuda_lib, 2, 1500, 300, 4, 2, 16, 32, t, lens=[300, 129])
    _check(cuda_lib, 1, 2100, 2100, 8, 1, 64, 128, t, causal=True, rms=ALL)


def test_lambda_in_fp32(cuda_lib):
    _check(cuda_lib, 1, 100, 100, 4, 2, 16, 32, BF16, lam_t=F32)


def test_large_scores_raise_the_maximum(cuda_lib):
    """Later keys exceed the running maximum by far more than the threshold of a rescale."""
    x = _inputs(1, 200, 700, 2, 2, 32, 64, BF16)
    for k in ("k1", "k2"):
        x[k] *= torch.linspace(0.1, 12, 700, device="cuda")[None, :, None, None].to(BF16)
    got = _run(cuda_lib, x, 32 ** -0.5, BF16)
    val, tol = _reference(x, 32 ** -0.5, BF16)
    _compare(got, val, tol, BF16)


def test_strided_views(cuda_lib):
    """q1 and q2 as halves of one projection, k1, k2 and v as heads of another: gradients go back the same way."""
    B, N, Hq, Hk, d, dv = 2, 100, 4, 2, 32, 64
    x = _inputs(B, N, N, Hq, Hk, d, dv, BF16)
    plain = _run(cuda_lib, x, d ** -0.5, BF16)
    bufs = {}

    def layout(k, v):
        if k == "lam":
            return v
        buf = torch.full((B + 1, N + 3, v.shape[2], 2, v.shape[3] + 8), 7.0, dtype=BF16, device="cuda")
        w = buf[:B, :N, :, 1, 8:]
        w.copy_(v)
        bufs.setdefault(k, []).append((buf, w))
        return w

    def st(h, e):
        return {"b": (N + 3) * h * 2 * (e + 8), "t": h * 2 * (e + 8), "h": 2 * (e + 8)}

    strides = {k: tuple(st(h, e).values()) for k, h, e in (("q_stride", Hq, d), ("k_stride", Hk, d), ("v_stride", Hk, dv), ("o_stride", Hq, dv))}
    got = _run(cuda_lib, x, d ** -0.5, BF16, strides=strides, layout=layout)
    for k in plain:
        assert torch.equal(plain[k], got[k]), k
    for pairs in bufs.values():
        for buf, w in pairs:       # nothing around the views was written
            w.fill_(7.0)
            assert bool((buf == 7.0).all())


def test_what_lies_behind_a_length_is_not_read(cuda_lib):
    x = _inputs(2, 40, 300, 2, 2, 16, 32, BF16)
    lens = torch.tensor([100, 17], dtype=torch.int32, device="cuda")
    one = _run(cuda_lib, x, 0.25, BF16, lens)
    for b, n in enumerate((100, 17)):
        for k in ("k1", "k2", "v"):
            x[k][b, n:] = float("nan")
    two = _run(cuda_lib, x, 0.25, BF16, lens)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_a_bad_score_spoils_its_row_alone(cuda_lib):
    x = _inputs(1, 200, 200, 1, 1, 16, 32, BF16)
    x["q1"][0, 3] = float("inf")
    x["q2"][0, 130, 0, 2] = float("nan")
    o = _run(cuda_lib, x, 0.25, BF16, train=False)["o"]
    bad = torch.isnan(o[0, :, 0]).all(1).nonzero()[:, 0].tolist()
    assert bad == [3, 130] and not torch.isnan(o).sum() > 2 * 32


def test_same_bits_twice_and_captured(cuda_lib):
    """Runs, replays and another stream agree to the bit, with a captured backward over its own workspaces."""
    rib, t = cuda_lib, BF16
    x = _inputs(2, 500, 500, 4, 2, 32, 64, t)
    one, two = (_run(rib, x, 0.2, t, causal=True) for _ in range(2))
    for k in one:
        assert torch.equal(one[k], two[k]), k
    desc = rib.diff_attn_desc(2, 500, 500, 4, 2, 32, 64, 0.2, t, causal=True)
    out = {k: torch.empty_like(v) for k, v in one.items()}
    ws = torch.empty(max(1, rib.rib_diff_attention_workspace_size(desc)), dtype=torch.uint8, device="cuda")
    wb = torch.empty(rib.rib_diff_attention_bwd_workspace_size(desc), dtype=torch.uint8, device="cuda")
    args = [x[k] for k in NAMES + ("lam",)] + [None]

    def step():
        rib.rib_diff_attention(desc, *args, out["o"], out["o2"], out["lse"], ws)
        rib.rib_diff_attention_bwd(desc, *args, out["o"], out["o2"], out["lse"], x["do"],
                                   *(out["d" + k] for k in NAMES + ("lam",)), wb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in out.values():
        v.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for k in one:
        assert torch.equal(one[k], out[k]), k


def test_empty_tensors(cuda_lib):
    rib = cuda_lib
    for B, Nq, Nk in ((0, 5, 5), (2, 0, 5), (2, 5, 0), (2, 0, 0)):
        x = _inputs(B, Nq, Nk, 4, 2, 16, 32, BF16)
        got = _run(rib, x, 0.25, BF16)
        for k, v in got.items():
            if k == "lse":
                assert bool((v == -math.inf).all())
            else:
                assert bool((v == 0).all()), (B, Nq, Nk, k)


def test_gradients_match_differences(cuda_lib):
    """The gradient against central differences of the fp64 loss at the kernel's rounded inputs."""
    B, N, Hq, Hk, d, dv, t = 1, 40, 2, 1, 16, 32, F16
    x = _inputs(B, N, N, Hq, Hk, d, dv, t)
    got = _run(cuda_lib, x, 0.25, t, causal=True)
    val, tol = _reference(x, 0.25, t, causal=True)
    g = torch.Generator().manual_seed(5)
    f = {k: v.double() for k, v in x.items()}
    for k in NAMES + ("lam",):
        step = torch.randn(x[k].shape, generator=g).double().cuda()
        h = 1e-5

        def loss(sign):
            y = dict(f)
            y[k] = f[k] + sign * h * step
            return float((_reference_o(y, 0.25) * f["do"]).sum())

        diff = (loss(1) - loss(-1)) / (2 * h)
        dot = float((got["d" + k].double() * step).sum())
        # the kernel's error bound along the step, and the difference's own: third order h^2 (1e-10 of order-one terms) and rounding 1e-10
        assert abs(dot - diff) <= float((tol["d" + k] * step.abs()).sum()) + 1e-5, k


def _reference_o(f, scale):
    Hq, Hk = f["q1"].shape[2], f["k1"].shape[2]
    r = lambda x: x.repeat_interleave(Hq // Hk, 2).transpose(1, 2)  # noqa: E731
    N = f["q1"].shape[1]
    hide = torch.ones(N, N, dtype=torch.bool, device="cuda").triu(1)
    a = [torch.softmax((f[q].transpose(1, 2) @ r(f[k]).transpose(2, 3) * scale).masked_fill(hide, -math.inf), -1)
         for q, k in (("q1", "k1"), ("q2", "k2"))]
    return ((a[0] - f["lam"][None, :, None, None] * a[1]) @ r(f["v"])).transpose(1, 2)


def test_a_training_block(cuda_lib):
    """h = norm(x), y = attention over windows, x' = x + dropout(scale norm(y)), next h, and back through all three,
    against autograd in fp64 from the kernels' own stored activations."""
    rib, t = cuda_lib, BF16
    H, W, heads, d, dv, window, p = 20, 26, 3, 16, 32, 8, 0.1
    T, C = H * W, heads * dv
    g = torch.Generator().manual_seed(9)
    n = lambda *s, dt=t: torch.randn(*s, generator=g).to(dt).cuda()  # noqa: E731
    x, scale = n(T, C, dt=F32), 0.5 + 0.1 * n(1, C, dt=F32)
    pw, pb = 1 + 0.1 * n(C, dt=F32), 0.1 * n(C, dt=F32)
    a = _inputs(1, T, T, heads, heads, d, dv, t)
    att = _run(rib, a, d ** -0.5, t, window=window, width=W, train=False)["o"].reshape(T, C)
    desc = rib.residual_norm_desc(T, C, F32, t, pre="layer", post="rms", p=p, seed=3, offset=1)
    x_out, h = torch.empty_like(x), torch.empty(T, C, dtype=t, device="cuda")
    rib.rib_residual_norm(desc, x, att, None, scale, None, None, pw, pb, x_out, h)
    dx_out, dh = n(T, C, dt=F32), n(T, C)
    dx, dy = torch.empty_like(x), torch.empty_like(att)
    rib.rib_residual_norm_bwd(desc, x_out, att, None, scale, None, None, pw, dx_out, dh, dx, dy)
    # the same join by autograd in fp64, its mask drawn by rib_dropout
    keep = torch.empty(T * C, device="cuda")
    rib.rib_dropout(torch.ones(T * C, device="cuda"), keep, p, 3, 1)
    xl, yl = x.double().requires_grad_(), att.double().requires_grad_()
    u = yl * torch.rsqrt(yl.square().mean(1, keepdim=True) + 1e-5)
    x1 = xl + keep.double().reshape(T, C) * scale.double() * u
    hl = torch.nn.functional.layer_norm(x1, (C,), pw.double(), pb.double(), 1e-5)
    gx, gy = torch.autograd.grad([x1, hl], [xl, yl], [dx_out.double(), dh.double()])
    assert (x_out.double() - x1).abs().max() <= 64 * 2.0 ** -24 * x1.abs().max()
    assert ((h.double() - hl).abs() <= 2.0 ** -8 * hl.abs() + 1e-4).all()
    assert ((dx.double() - gx).abs() <= 1e-4).all()           # fp32 all the way
    # r of a branch row is at most 1 / min rms of y; fp32 terms of that size, then bf16
    ry = float((1 / att.double().square().mean(1).sqrt()).max())
    assert ((dy.double() - gy).abs() <= 2.0 ** -8 * gy.abs() + 256 * 2.0 ** -24 * ry * gx.abs().max() * 8).all()
    # and the attention's backward from that gradient
    a["do"] = dy.reshape(1, T, heads, dv)
    got = _run(rib, a, d ** -0.5, t, window=window, width=W)
    val, tol = _reference(a, d ** -0.5, t, window=window, width=W)
    _compare(got, val, tol, t)


@pytest.mark.parametrize("t", [F16, BF16])
@pytest.mark.parametrize("d,dv", [(16, 32), (64, 128)])
def test_small_scales(cuda_lib, d, dv, t):
    """lse / scale far beyond fp16 (2^-8 of it is 2e5 here): large queries and keys under a scale of 2e-8."""
    x = _inputs(1, 150, 190, 2, 1, d, dv, t)
    for k in ("q1", "q2", "k1", "k2"):
        x[k] *= 1500 * (64 / d) ** 0.25
    x["do"] *= 256          # keeps the gradients of q and k among fp16's normal values
    got = _run(cuda_lib, x, 2e-8, t)
    val, tol = _reference(x, 2e-8, t)
    _compare(got, val, tol, t, rms=ALL)


def test_huge_scores(cuda_lib):
    """Scores of millions: lse / scale is the raw score, above 2^24. Each row's own key outweighs all others."""
    x = _inputs(1, 70, 70, 1, 1, 64, 128, F16)
    for k in ("q1", "q2"):
        x[k].copy_(torch.where(x[k] > 0, 600.0, -600.0))
    for k in ("k1", "k2"):
        x[k].copy_(x["q" + k[1]])
    got = _run(cuda_lib, x, 0.125, F16)
    # the own key scores 2.9e6 and the next 1e6 less: both maps are one-hot, o = (1 - lam) v. P is rounded (u) and so is o
    lam, u, low = x["lam"].double(), torch.finfo(F16).eps / 2, 2.0 ** -24
    v, do = x["v"].double().abs(), x["do"].double().abs()
    assert ((got["o"].double() - (1 - lam) * x["v"].double()).abs() <= 3 * u * (1 + lam.abs()) * v + low).all()
    # the log-sum-exp, 4.2e6 in powers of two, passes seven fp32 roundings of 2^-2 on its way into the backward's P: a factor
    # of 2^1.75 at most. Nothing is lost beyond that: dv is P dO, and dP - D what the roundings of P, o and o2 leave
    f = 2 ** 1.75 * (1 + 4 * u)
    assert (got["dv"].double().abs() <= f * (1 + lam.abs()) * do + low).all()
    e = f * (1 + lam.abs()) * 8 * u * (do * v).sum(-1).max()
    for k in ("dq1", "dq2", "dk1", "dk2"):
        assert (got[k].double().abs() <= 0.125 * 600 * e).all(), k


def test_infinite_scores(cuda_lib):
    """Scores that overflow fp32: -infinity is a key that the row does not see, in both directions; +infinity spoils the row."""
    t, N, r, h = BF16, 200, 3, 0
    x = _inputs(1, N, N, 1, 1, 16, 32, t)
    x["q1"][..., 0] = 0
    x["k1"][..., 0] = -1e20
    x["do"][0, r] = 0
    want = _run(cuda_lib, x, 0.25, t)
    g = torch.Generator().manual_seed(3)
    x["do"][0, r] = torch.randn(1, 32, generator=g).to(t).cuda()
    # every key of row r's first map scores -1e40: the map is empty, and has no part in any gradient
    x["q1"][0, r, h, 0] = 1e20
    got = _run(cuda_lib, x, 0.25, t)
    others = torch.arange(N, device="cuda") != r
    assert bool((got["lse"][0, 0, h, r] == -math.inf).all()) and torch.equal(got["lse"][1], want["lse"][1])
    assert torch.equal(got["lse"][0][..., others], want["lse"][0][..., others])
    for k in ("o", "o2", "dq1", "dq2"):
        assert torch.equal(got[k][0, others], want[k][0, others]), k
    u = torch.finfo(t).eps / 2
    o, o2, lam = got["o"][0, r].double(), got["o2"][0, r].double(), x["lam"].double()
    assert ((o + lam * o2).abs() <= 2 * u * (lam * o2).abs() + 1e-30).all()      # o and o2 are each rounded
    assert bool((got["dq1"][0, r] == 0).all()) and torch.equal(got["dk1"], want["dk1"])
    assert torch.isfinite(got["dk2"]).all() and torch.isfinite(got["dv"]).all() and bool((got["dq2"][0, r] != 0).any())
    # some of them do: the row is the softmax over the rest
    x["k1"][0, 100:, h, 0] = 0
    got = _run(cuda_lib, x, 0.25, t)
    a = [torch.softmax((x[q][0, r, h].double() @ x[k][0, at:, h].double().T * 0.25), -1) for q, k, at in (("q1", "k1", 100), ("q2", "k2", 0))]
    v = x["v"][0, :, h].double()
    ref, mag = a[0] @ v[100:] - lam * (a[1] @ v), a[0] @ v[100:].abs() + lam.abs() * (a[1] @ v.abs())
    assert ((got["o"][0, r, h].double() - ref).abs() <= (u + 2.0 ** -16) * mag + u * ref.abs()).all()
    for k in ("dq1", "dq2", "dk1", "dk2", "dv", "dlam"):
        assert torch.isfinite(got[k]).all(), k
    # and +infinity
    x["q1"][0, 130, h, 0] = -1e20
    o = _run(cuda_lib, x, 0.25, t, train=False)["o"]
    assert torch.isnan(o[0, :, h]).all(1).nonzero()[:, 0].tolist() == [130] and int(torch.isnan(o).sum()) == 32


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("d,dv", [(64, 128), (48, 104), (64, 64), (24, 40)])
@pytest.mark.parametrize("H,W,window,Hq,Hk", [(13, 29, 8, 2, 2), (40, 33, 31, 2, 1), (20, 70, 64, 4, 2), (9, 7, 16, 3, 1)])
def test_windows_of_every_width_class(cuda_lib, H, W, window, Hq, Hk, d, dv, t):
    """Cut boxes and shared heads with one score buffer in the key-side kernel (dv above 64) and with two."""
    _check(cuda_lib, 2, H * W, H * W, Hq, Hk, d, dv, t, window=window, width=W)


@pytest.mark.parametrize("d,dv", [(64, 128), (32, 64)])
def test_a_bad_window_stays_in_its_window_at_wide_heads(cuda_lib, d, dv):
    t, H, W, window = BF16, 26, 29, 12
    x = _inputs(1, H * W, H * W, 2, 1, d, dv, t)
    one = _run(cuda_lib, x, 0.125, t, window=window, width=W)
    bad = torch.zeros(H, W, dtype=torch.bool, device="cuda")
    bad[window:2 * window, :window] = True
    bad = bad.reshape(-1)
    for k in NAMES + ("do",):
        x[k][0, bad] = float("nan")
    two = _run(cuda_lib, x, 0.125, t, window=window, width=W)
    for k in ("o", "o2", "dq1", "dq2", "dk1", "dk2", "dv"):
        assert torch.equal(one[k][0, ~bad], two[k][0, ~bad]), k
        assert torch.isnan(two[k][0, bad]).all(), k
    assert torch.equal(one["lse"][..., ~bad], two["lse"][..., ~bad])


@pytest.mark.parametrize("t", [BF16, F16])
@pytest.mark.parametrize("B,Nq,Nk,Hq,Hk,d,dv,kw", [
    (2, 150, 190, 2, 2, 16, 32, {}), (2, 150, 190, 4, 2, 64, 128, {"causal": True}), (2, 3, 4099, 8, 2, 64, 128, {}), (1, 70, 6000, 1, 1, 32, 64, {}),
    (2, 35 * 22, 35 * 22, 2, 1, 24, 40, {"window": 16, "width": 22})], ids=["two-groups", "one-group", "few-rows", "split", "windows"])
def test_a_bad_query_spoils_its_row_in_every_form(cuda_lib, B, Nq, Nk, Hq, Hk, d, dv, kw, t):
    """A NaN query makes its row of o NaN, in either map, and leaves every other row's bits."""
    x = _inputs(B, Nq, Nk, Hq, Hk, d, dv, t)
    one = _run(cuda_lib, x, 0.125, t, train=False, **kw)["o"]
    rows = [(0, Nq // 2, 0), (B - 1, Nq - 1, Hq - 1)]
    for k, (b, n, h) in zip(("q1", "q2"), rows):
        x[k][b, n, h, d - 1] = float("nan")
    two = _run(cuda_lib, x, 0.125, t, train=False, **kw)["o"]
    bad = torch.zeros(B, Nq, Hq, dtype=torch.bool, device="cuda")
    for r in rows:
        bad[r] = True
    assert torch.isnan(two[bad]).all() and torch.equal(one[~bad], two[~bad])
