"""Cases and plain forms of the training-block operators around the windowed attention.

Three operators, each with a plain form in elementary torch operations and with the call a user makes of the package:

* ``norm``: the join of a block with its residual stream. With u = N_post(y) post_w + post_b,
  x' = x + dropout(scale * gate * u) and h = N_pre(x') pre_w + pre_b, N one of LayerNorm, RMSNorm or nothing;
  scale is one row of C values per group of rows (one group: a residual scale; one per image: a per-image gate).
* ``dropout``: y = x / keep where the element's 16 random bits reach the threshold, 0 elsewhere. The bits come from
  Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", SC 2011) at counter
  (element // 8, offset) and key seed, eight elements a call, so no mask is ever stored.
* ``attn``: differential attention, O = (softmax(s q1 k1^T) - lambda softmax(s q2 k2^T)) v, over the windows of a map or
  over sequences, with shared key heads, key lengths and a causal mask.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


# ---------------------------------------------------------------------- cases
def _norm(rows, cols, residual="f32", dtype="bf16", pre="layer", post="layer", gate=True, groups=1, p=0.0, train=False):
    return {"op": "norm", "rows": rows, "cols": cols, "residual": residual, "dtype": dtype, "pre": pre, "post": post,
            "gate": gate, "groups": groups, "p": p, "train": train}


def _drop(n, dtype, p, train=False):
    return {"op": "dropout", "n": n, "dtype": dtype, "p": p, "train": train}


def _attn(batch, q_len, k_len, heads, kv_heads, d, dv, dtype="bf16", causal=False, ragged=False, width=0, window=0, train=False):
    return {"op": "attn", "batch": batch, "q_len": q_len, "k_len": k_len, "heads": heads, "kv_heads": kv_heads, "d": d,
            "dv": dv, "dtype": dtype, "causal": causal, "ragged": ragged, "width": width, "window": window, "train": train}


def listed():
    return [
        # one 8x8 patch of the lite width: the call's own latency
        {"name": "norm 8x8 patch", **_norm(64, 48)},
        # the 640x360 map of the full layer, inference
        {"name": "norm 640x360 map", **_norm(360 * 640, 180)},
        # 16 patches of 96x96, a training step with residual dropout
        {"name": "norm train 16x96x96", **_norm(16 * 96 * 96, 180, p=0.1, train=True)},
        # a wide odd channel count, RMS norms, one scale row per image, fp16 branch
        {"name": "norm train odd width", **_norm(7 * 577, 1021, dtype="f16", pre="rms", post="rms", groups=7, train=True)},
        # a small activation map
        {"name": "dropout 16x16x48", **_drop(16 * 16 * 48, "bf16", 0.1)},
        # the whole 640x360x180 map, forward and backward
        {"name": "dropout train map", **_drop(360 * 640 * 180, "bf16", 0.1, train=True)},
        # fp32 activations with a ragged end
        {"name": "dropout f32 odd", **_drop(180 * 320 * 48 + 3, "f32", 0.25)},
        # the tiny layer's map: four windows of 16x16
        {"name": "attn 32x32 window 16", **_attn(1, 32 * 32, 32 * 32, 3, 3, 16, 32, width=32, window=16)},
        # the lite map with the full layer's heads: the last row of windows is cut at 52 of 64 rows
        {"name": "attn 320x180 window 64", **_attn(1, 320 * 180, 320 * 180, 6, 6, 16, 32, width=320, window=64)},
        # training patches, one window each
        {"name": "attn train 2x96x96", **_attn(2, 96 * 96, 96 * 96, 6, 6, 16, 32, width=96, window=96, train=True)},
        # causal sequences with shared key heads and wide heads
        {"name": "attn train causal", **_attn(2, 4001, 4001, 8, 2, 64, 128, causal=True, train=True)},
        # one new token per sequence over a long cache of ragged lengths
        {"name": "attn single token", **_attn(16, 1, 8192, 16, 4, 64, 128, ragged=True)},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "dropout", "attn", "attn", "attn"])
    if op == "norm":
        cols = rng.choice([_log(rng, 8, 4096), 4 * _log(rng, 8, 256)])
        groups = rng.choice([1, 1, 2, 5])
        rows = groups * _log(rng, 1, max(2, 36_000_000 // (cols * groups)))
        dtype = rng.choice(["bf16", "f16"])
        train = rng.random() < 0.5
        residual = "f32" if train else rng.choice(["f32", dtype])
        pre = rng.choice(["layer", "rms"])
        post = rng.choice(["layer", "rms", "none"])
        return _norm(rows, cols, residual, dtype, pre, post, rng.random() < 0.5, groups, rng.choice([0.0, 0.1, 0.35]), train)
    if op == "dropout":
        return _drop(_log(rng, 1000, 40_000_000), rng.choice(["bf16", "f16", "f32"]), rng.choice([0.05, 0.1, 0.25, 0.5]), rng.random() < 0.5)
    while True:  # a drawn case costs no more than the largest listed one
        c = _draw_attn(rng)
        if _pairs(c) * c["heads"] <= 1.0e9 and work(c)["flops"] <= 5.0e11:
            return c


def _draw_attn(rng):
    d, dv = rng.choice([(16, 32), (24, 40), (32, 64), (64, 64), (64, 128)])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    kind = rng.choice(["window", "train", "single"])
    if kind == "window":
        window = rng.choice([8, 12, 16, 31, 32, 48, 64])
        height, width = rng.randint(window, 4 * window), rng.randint(window, 4 * window)
        heads = rng.choice([1, 3, 6])
        return _attn(rng.choice([1, 2]), height * width, height * width, heads, heads, d, dv, dtype, width=width, window=window,
                     train=rng.random() < 0.5)
    if kind == "train":
        kv = rng.choice([1, 2, 3])
        n = _log(rng, 33, 2900)
        return _attn(rng.choice([1, 2]), n, n, kv * rng.choice([1, 2, 4]), kv, d, dv, dtype, causal=rng.random() < 0.5, train=True)
    kv = rng.choice([1, 4])
    return _attn(_log(rng, 1, 32), rng.choice([1, 1, 4]), _log(rng, 64, 16384), kv * rng.choice([1, 4, 8]), kv, d, dv, dtype, ragged=True)


# --------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, mul=1.0, add=0.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(mul).add_(add).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case, "seed": (seed * 0x9E3779B97F4A7C15 + 1) % (1 << 64), "offset": seed % 1000}
    if case["op"] == "dropout":
        t = DTYPES[case["dtype"]]
        st["x"] = _randn(g, case["n"], dtype=t)
        st["y"] = torch.empty_like(st["x"])
        if case["train"]:
            st["dy"], st["dx"] = _randn(g, case["n"], dtype=t), torch.empty_like(st["x"])
        return st
    if case["op"] == "norm":
        T, C, xt, t = case["rows"], case["cols"], DTYPES[case["residual"]], DTYPES[case["dtype"]]
        st["x"], st["y"] = _randn(g, T, C, dtype=xt), _randn(g, T, C, dtype=t, mul=1.5, add=0.1)
        st["gate"] = torch.sigmoid(_randn(g, T, C)).to(t) if case["gate"] else None
        st["scale"] = _randn(g, case["groups"], C, mul=0.1, add=0.5)
        for k, n in (("post", case["post"]), ("pre", case["pre"])):
            st[k + "_w"] = _randn(g, C, mul=0.1, add=1.0) if n != "none" else None
            st[k + "_b"] = _randn(g, C, mul=0.1) if n == "layer" else None
        st["x_out"], st["h"] = torch.empty_like(st["x"]), torch.empty_like(st["y"])
        if case["train"]:
            st["dx_out"], st["dh"] = _randn(g, T, C, dtype=xt), _randn(g, T, C, dtype=t)
            for k in ("x", "y", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b"):
                st["d" + k] = None if st[k] is None else torch.empty_like(st[k])
        return st
    B, Nq, Nk, Hq, Hk, d, dv = (case[k] for k in ("batch", "q_len", "k_len", "heads", "kv_heads", "d", "dv"))
    t = DTYPES[case["dtype"]]
    for k, n, h, e in (("q1", Nq, Hq, d), ("q2", Nq, Hq, d), ("k1", Nk, Hk, d), ("k2", Nk, Hk, d), ("v", Nk, Hk, dv)):
        st[k] = _randn(g, B, n, h, e, dtype=t)
    st["lam"] = (0.2 + 0.6 * torch.rand(Hq, generator=g, device="cuda")).to(t)
    st["k_lens"] = torch.randint(Nk // 2, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
    st["o"] = torch.empty(B, Nq, Hq, dv, dtype=t, device="cuda")
    if case["train"]:
        st["do"] = _randn(g, B, Nq, Hq, dv, dtype=t)
        st["o2"], st["lse"] = torch.empty_like(st["o"]), torch.empty(2, B, Hq, Nq, device="cuda")
        for k in ("q1", "q2", "k1", "k2", "v", "lam"):
            st["d" + k] = torch.empty_like(st[k])
    return st


# ------------------------------------------------------------------ plain forms
def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _keep_mask(n, p, seed, offset):
    """True where the element is kept, and 1 / (kept share)."""
    low = 0xFFFFFFFF
    at = torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64)
    c0, c1 = at & low, at >> 32
    c2, c3 = torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)
    k0, k1 = seed & low, seed >> 32

    def high(m, v):  # upper 32 bits of m * v by 16-bit halves, which 63 bits hold
        return (m * (v >> 16) + ((m * (v & 0xFFFF)) >> 16)) >> 16

    for _ in range(10):
        h0, l0 = high(0xD2511F53, c0), (0xD2511F53 * c0) & low
        h1, l1 = high(0xCD9E8D57, c2), (0xCD9E8D57 * c2) & low
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 1)
    bits = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n]
    thr = _threshold(p)
    return bits >= thr, 65536.0 / (65536 - thr) if thr < 65536 else 0.0


def _stats(x, kind):
    """(x - mean) * rstd and rstd over the last axis."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_grad(t, xhat, r, kind):
    """Gradient at the norm's input from t, the gradient at xhat."""
    t = t - xhat * (t * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    return t * r


def _by_group(m, groups):
    return m.reshape(groups, -1, m.shape[-1]).sum(1)


def _norm_plain(st):
    c = st["case"]
    T, C, G = c["rows"], c["cols"], c["groups"]
    xt, t = DTYPES[c["residual"]], DTYPES[c["dtype"]]
    x, y = st["x"].float(), st["y"].float()
    yhat, ry = _stats(y, c["post"]) if c["post"] != "none" else (y, None)
    u = yhat * st["post_w"] if c["post"] != "none" else yhat
    u = u + st["post_b"] if st["post_b"] is not None else u
    f = st["scale"].repeat_interleave(T // G, 0)
    if c["p"]:
        keep, up = _keep_mask(T * C, c["p"], st["seed"], st["offset"])
        f = torch.where(keep.reshape(T, C), f * up, 0.0)
    fg = f * st["gate"].float() if c["gate"] else f
    x1 = x + fg * u
    xhat, rx = _stats(x1, c["pre"])
    h = xhat * st["pre_w"]
    h = h + st["pre_b"] if st["pre_b"] is not None else h
    out = {"x_out": x1.to(xt), "h": h.to(t)}
    if not c["train"]:
        return out
    dh = st["dh"].float()
    dx = st["dx_out"].float() + _norm_grad(dh * st["pre_w"], xhat, rx, c["pre"])
    out["dx"] = dx.to(xt)
    out["dpre_w"] = (dh * xhat).sum(0)
    if st["pre_b"] is not None:
        out["dpre_b"] = dh.sum(0)
    if c["gate"]:
        out["dgate"] = (dx * f * u).to(t)
    part = dx * u * st["gate"].float() if c["gate"] else dx * u
    if c["p"]:
        part = torch.where(keep.reshape(T, C), part * up, 0.0)
    out["dscale"] = _by_group(part, G)
    du = dx * fg
    if c["post"] == "none":
        out["dy"] = du.to(t)
        return out
    out["dpost_w"] = (du * yhat).sum(0)
    if st["post_b"] is not None:
        out["dpost_b"] = du.sum(0)
    out["dy"] = _norm_grad(du * st["post_w"], yhat, ry, c["post"]).to(t)
    return out


def _windows(case):
    """Token numbers of each window [windows, window^2], -1 behind the map's edge."""
    M, W = case["window"], case["width"]
    H = case["q_len"] // W
    wy, wx = -(-H // M), -(-W // M)
    y = torch.arange(wy * M, device="cuda").reshape(wy, 1, M, 1)
    x = torch.arange(wx * M, device="cuda").reshape(1, wx, 1, M)
    at = torch.where((y < H) & (x < W), y * W + x, -1)
    return at.reshape(wy * wx, M * M)


def _split(x, at):
    """[batch, tokens, heads, e] -> [batch * windows, heads, window^2, e] in 32 bits, zeros behind the edge."""
    if at is None:
        return x.float().transpose(1, 2)
    y = x.float()[:, at.clamp(min=0)]
    y = y * (at >= 0)[None, :, :, None, None]
    return y.flatten(0, 1).transpose(1, 2)


def _merge(x, at, like):
    """The inverse of _split, rounded to the type of `like`."""
    if at is None:
        return x.transpose(1, 2).to(like.dtype)
    y = x.transpose(1, 2).reshape(like.shape[0], *at.shape, *like.shape[2:])
    out = torch.empty(like.shape, dtype=torch.float32, device="cuda")
    out[:, at[at >= 0]] = y[:, at >= 0]
    return out.to(like.dtype)


def _softmax(s, seen):
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -math.inf, m, 0.0))
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, 1.0)


def _attn_plain(st):
    c = st["case"]
    G = c["heads"] // c["kv_heads"]
    at = _windows(c) if c["window"] else None
    q1, q2 = _split(st["q1"], at), _split(st["q2"], at)
    k1, k2, v = (_split(st[k], at).repeat_interleave(G, 1) for k in ("k1", "k2", "v"))
    if at is not None:
        seen = (at >= 0).repeat(c["batch"], 1)[:, None, None, :]
    else:
        j = torch.arange(c["k_len"], device="cuda")
        lens = st["k_lens"] if c["ragged"] else torch.full((c["batch"],), c["k_len"], device="cuda")
        seen = (j < lens[:, None])[:, None, None, :]
        if c["causal"]:
            i = torch.arange(c["q_len"], device="cuda")
            seen = seen & (j <= i[:, None] + (lens[:, None, None, None] - c["q_len"]))
    scale, lam = c["d"] ** -0.5, st["lam"].float()[:, None, None]
    a1 = _softmax(q1 @ k1.transpose(2, 3) * scale, seen)
    a2 = _softmax(q2 @ k2.transpose(2, 3) * scale, seen)
    o2 = a2 @ v
    out = {"o": _merge(a1 @ v - lam * o2, at, st["o"])}
    if not c["train"]:
        return out
    do = _split(st["do"], at)
    dlam = -(do * o2).sum((0, 2, 3))
    dv = (a1 - lam * a2).transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    shared = lambda x: x.unflatten(1, (c["kv_heads"], G)).sum(2)  # noqa: E731
    ds = a1 * (dp - (a1 * dp).sum(-1, keepdim=True)) * scale
    out["dq1"], out["dk1"] = _merge(ds @ k1, at, st["q1"]), _merge(shared(ds.transpose(2, 3) @ q1), at, st["k1"])
    del a1, ds
    ds = -lam * a2 * (dp - (a2 * dp).sum(-1, keepdim=True)) * scale
    out["dq2"], out["dk2"] = _merge(ds @ k2, at, st["q2"]), _merge(shared(ds.transpose(2, 3) @ q2), at, st["k2"])
    out["dv"], out["dlam"] = _merge(shared(dv), at, st["v"]), dlam.to(st["lam"].dtype)
    return out


def _dropout_plain(st):
    c = st["case"]
    keep, up = _keep_mask(c["n"], c["p"], st["seed"], st["offset"])
    f = torch.where(keep, up, 0.0)
    out = {"y": (st["x"].float() * f).to(st["x"].dtype)}
    if c["train"]:
        out["dx"] = (st["dy"].float() * f).to(st["x"].dtype)
    return out


# ------------------------------------------------------------ the package's calls
def _norm_own(st):
    import windowed_attention_b200 as rib
    c = st["case"]
    if "desc" not in st:
        st["desc"] = rib.residual_norm_desc(c["rows"], c["cols"], st["x"].dtype, st["y"].dtype, pre=c["pre"], post=c["post"], eps=EPS,
                                            rows_per_group=c["rows"] // c["groups"], p=c["p"], seed=st["seed"], offset=st["offset"])
        n = rib.rib_residual_norm_bwd_workspace_size(st["desc"]) if c["train"] else 0
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    rib.rib_residual_norm(st["desc"], st["x"], st["y"], st["gate"], st["scale"], st["post_w"], st["post_b"], st["pre_w"], st["pre_b"],
                          st["x_out"], st["h"])
    out = {"x_out": st["x_out"], "h": st["h"]}
    if c["train"]:
        rib.rib_residual_norm_bwd(st["desc"], st["x_out"], st["y"], st["gate"], st["scale"], st["post_w"], st["post_b"], st["pre_w"],
                                  st["dx_out"], st["dh"], st["dx"], st["dy"], st["dgate"], st["dscale"], st["dpost_w"], st["dpost_b"],
                                  st["dpre_w"], st["dpre_b"], st["ws"])
        for k in ("dx", "dy", "dgate", "dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b"):
            if st[k] is not None:
                out[k] = st[k]
    return out


def _dropout_own(st):
    import windowed_attention_b200 as rib
    c = st["case"]
    rib.rib_dropout(st["x"], st["y"], c["p"], st["seed"], st["offset"])
    out = {"y": st["y"]}
    if c["train"]:
        rib.rib_dropout(st["dy"], st["dx"], c["p"], st["seed"], st["offset"])
        out["dx"] = st["dx"]
    return out


def _attn_own(st):
    import windowed_attention_b200 as rib
    c = st["case"]
    if "desc" not in st:
        st["desc"] = rib.diff_attn_desc(c["batch"], c["q_len"], c["k_len"], c["heads"], c["kv_heads"], c["d"], c["dv"], c["d"] ** -0.5,
                                        dtype=st["q1"].dtype, causal=c["causal"], width=c["width"], window=c["window"])
        n = rib.rib_diff_attention_workspace_size(st["desc"])
        n = max(n, rib.rib_diff_attention_bwd_workspace_size(st["desc"])) if c["train"] else n
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    qkv = [st[k] for k in ("q1", "q2", "k1", "k2", "v", "lam", "k_lens")]
    if not c["train"]:
        rib.rib_diff_attention(st["desc"], *qkv, st["o"], None, None, st["ws"])
        return {"o": st["o"]}
    rib.rib_diff_attention(st["desc"], *qkv, st["o"], st["o2"], st["lse"], st["ws"])
    grads = [st["d" + k] for k in ("q1", "q2", "k1", "k2", "v", "lam")]
    rib.rib_diff_attention_bwd(st["desc"], *qkv, st["o"], st["o2"], st["lse"], st["do"], *grads, st["ws"])
    return {"o": st["o"], **{"d" + k: x for k, x in zip(("q1", "q2", "k1", "k2", "v", "lam"), grads)}}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "dropout": _dropout_own, "attn": _attn_own}[op](state)
    return {"norm": _norm_plain, "dropout": _dropout_plain, "attn": _attn_plain}[op](state)


# ------------------------------------------------------------------------ work
def _pairs(c):
    """(query, key) pairs of one head that a mask without lengths leaves, keys counted in full where they are ragged."""
    if c["window"]:
        M, W = c["window"], c["width"]
        H = c["q_len"] // W
        ys = [min(M, H - y) for y in range(0, H, M)]
        xs = [min(M, W - x) for x in range(0, W, M)]
        return c["batch"] * sum(y * y for y in ys) * sum(x * x for x in xs)
    if c["causal"]:
        return c["batch"] * sum(max(0, min(c["k_len"], i + 1 + c["k_len"] - c["q_len"])) for i in range(c["q_len"]))
    return c["batch"] * c["q_len"] * c["k_len"] * (0.75 if c["ragged"] else 1)


def work(case):
    if case["op"] == "dropout":
        b = 2 * case["n"] * SIZES[case["dtype"]] * (2 if case["train"] else 1)
        return {"bytes": b, "flops": 2 * case["n"]}
    if case["op"] == "norm":
        n, x, t = case["rows"] * case["cols"], SIZES[case["residual"]], SIZES[case["dtype"]]
        g = 1 if case["gate"] else 0
        b = n * (2 * x + 2 * t + g * t)
        if case["train"]:  # reads dx', dh, writes dx, dy and the gate's gradient
            b += n * (2 * x + 2 * t + g * t)
        return {"bytes": b, "flops": n * (60 if case["train"] else 20)}
    B, Nq, Nk, Hq, Hk, d, dv = (case[k] for k in ("batch", "q_len", "k_len", "heads", "kv_heads", "d", "dv"))
    q, k = 2 * B * Nq * Hq, 2 * B * Nk * Hk * (0.75 if case["ragged"] else 1)
    b = q * (2 * d + dv) + k * (2 * d + dv)
    f = _pairs(case) * Hq * 4 * (d + dv)
    if case["train"]:
        b += q * (2 * d + dv) + k * (2 * d + dv)
        f += _pairs(case) * Hq * (12 * d + 4 * dv)
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------- definition in 64 bits
def _bits(n, seed, offset):
    """The 16 random bits of each element, from numpy's unsigned 64-bit products."""
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = [block & low, block >> s, np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(b >> s) ^ ctr[1] ^ np.uint64(key[0]), b & low, (a >> s) ^ ctr[3] ^ np.uint64(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(ctr, 1).astype("<u4").view("<u2").reshape(-1)[:n].astype(np.int32)


def _factor(case, st, n):
    """0 or 1 / keep for each element, in 64 bits on the GPU."""
    thr = _threshold(case["p"])
    bits = torch.from_numpy(_bits(n, st["seed"], st["offset"])).cuda()
    return (bits >= thr).double() * (65536.0 / (65536 - thr))


def _exact_norm(case, st):
    """Gradients by differentiating the definition."""
    T, C = case["rows"], case["cols"]
    leaf = {k: st[k].double().requires_grad_() for k in ("x", "y", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b") if st[k] is not None}

    def normed(x, kind, name):
        if kind == "none":
            return x
        if kind == "layer":
            var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
            x = (x - mean) / torch.sqrt(var + EPS)
        else:
            x = x / torch.sqrt((x * x).sum(1, keepdim=True) / C + EPS)
        x = leaf[name + "_w"] * x
        return x + leaf[name + "_b"] if name + "_b" in leaf else x

    with torch.enable_grad():
        r = normed(leaf["y"], case["post"], "post").reshape(case["groups"], -1, C) * leaf["scale"][:, None]
        r = r.reshape(T, C)
        if case["gate"]:
            r = r * leaf["gate"]
        if case["p"]:
            r = r * _factor(case, st, T * C).reshape(T, C)
        x1 = leaf["x"] + r
        h = normed(x1, case["pre"], "pre")
        out = {"x_out": x1.detach(), "h": h.detach()}
        if case["train"]:
            grads = torch.autograd.grad([x1, h], list(leaf.values()), [st["dx_out"].double(), st["dh"].double()])
            out.update({"d" + k: g for k, g in zip(leaf, grads)})
    return out


def _exact_attn(case, st):
    """One sequence and head at a time, the maps in full."""
    B, Hq = case["batch"], case["heads"]
    G, scale, train = Hq // case["kv_heads"], 1 / math.sqrt(case["d"]), case["train"]
    names = ("q1", "q2", "k1", "k2", "v")
    x = {k: st[k].double() for k in names + (("do",) if train else ())}
    out = {"o": torch.zeros_like(st["o"], dtype=torch.float64)}
    if train:
        out.update({"d" + k: torch.zeros_like(x[k]) for k in names})
        out["dlam"] = torch.zeros(Hq, dtype=torch.float64, device="cuda")
    lam = st["lam"].double()
    rows = [r[r >= 0] for r in _windows(case)] if case["window"] else [slice(None)]
    for b in range(B):
        n = int(st["k_lens"][b]) if case["ragged"] else case["k_len"]
        for r in rows:
            for h in range(Hq):
                kr = r if case["window"] else slice(0, n)
                g = h // G
                q1, q2, k1, k2, v = x["q1"][b, r, h], x["q2"][b, r, h], x["k1"][b, kr, g], x["k2"][b, kr, g], x["v"][b, kr, g]
                s1, s2 = q1 @ k1.T * scale, q2 @ k2.T * scale
                if case["causal"]:
                    hide = torch.ones_like(s1, dtype=torch.bool).triu(1 + n - case["q_len"])
                    s1, s2 = s1.masked_fill_(hide, -math.inf), s2.masked_fill_(hide, -math.inf)
                a1, a2 = torch.softmax(s1, 1), torch.softmax(s2, 1)
                del s1, s2
                out["o"][b, r, h] = a1 @ v - lam[h] * (a2 @ v)
                if not train:
                    continue
                do = x["do"][b, r, h]
                da = do @ v.T
                out["dlam"][h] -= (a2 * da).sum()
                out["dv"][b, kr, g] += a1.T @ do - lam[h] * (a2.T @ do)
                for a, q, k, nq, nk, f in ((a1, q1, k1, "dq1", "dk1", scale), (a2, q2, k2, "dq2", "dk2", -lam[h] * scale)):
                    ds = a * da
                    ds -= a * ds.sum(1, keepdim=True)
                    ds *= f
                    out[nq][b, r, h] = ds @ k
                    out[nk][b, kr, g] += ds.T @ q
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    if case["op"] == "attn":
        return _exact_attn(case, st)
    f = _factor(case, st, case["n"])
    out = {"y": st["x"].double() * f}
    if case["train"]:
        out["dx"] = st["dy"].double() * f
    return out
