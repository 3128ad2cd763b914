"""Plain fp64 NumPy oracle of the training-block operators: the residual join
with its norms, counter-based dropout and differential attention, forward and
backward from their formulas. Used only by tests."""
from __future__ import annotations

import numpy as np

M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox4x32_10(counter, key):
    """The four output words of Philox4x32-10 (Salmon et al., SC 2011) for
    counters [n, 4] and one key (two 32-bit words)."""
    c = [np.asarray(counter, np.uint64)[:, i] for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(M0), c[2] * np.uint64(M1)
        c = [(b >> s) ^ c[1] ^ np.uint64(k0), b & low, (a >> s) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + W0) & 0xFFFFFFFF, (k1 + W1) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def dropout_factor(n, p, seed, offset, first=0):
    """Factors 0 or 1/keep of elements first .. first + n - 1 (first a multiple of 8)."""
    thr = int(np.floor(p * 65536 + 0.5))
    blocks = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(first // 8)
    low = np.uint64(0xFFFFFFFF)
    ctr = np.stack([blocks & low, blocks >> np.uint64(32), np.full_like(blocks, offset & 0xFFFFFFFF),
                    np.full_like(blocks, (offset >> 32) & 0xFFFFFFFF)], 1)
    w = philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    bits = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:n]
    return np.where(bits >= thr, 65536.0 / max(1, 65536 - thr), 0.0)


def _normed(v, kind, eps):
    if kind == "none":
        return v, None
    d = v - v.mean(1, keepdims=True) if kind == "layer" else v
    r = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return d * r, r


def _normed_bwd(t, vh, r, kind):
    if kind == "none":
        return t
    t = t - vh * (t * vh).mean(1, keepdims=True)
    if kind == "layer":
        t = t - t.mean(1, keepdims=True)
    return r * t


def _or(v, other):
    return other if v is None else v


def residual_norm(x, y=None, gate=None, scale=None, post_w=None, post_b=None, pre_w=None, pre_b=None, pre="layer",
                  post="none", eps=1e-5, rows_per_group=None, mask=None):
    """(x_out, h); scale [groups, C], mask the dropout factors [T, C]."""
    x1 = x
    if y is not None:
        u = _normed(y, post, eps)[0] * _or(post_w, 1.0) + _or(post_b, 0.0)
        x1 = x + _or(mask, 1.0) * _rows(scale, x.shape[0], rows_per_group) * _or(gate, 1.0) * u
    h = None
    if pre != "none":
        h = _normed(x1, pre, eps)[0] * _or(pre_w, 1.0) + _or(pre_b, 0.0)
    return x1, h


def _rows(scale, T, rows_per_group):
    if scale is None:
        return 1.0
    return scale[np.arange(T) // (rows_per_group or T)]


def residual_norm_bwd(x_out, y=None, gate=None, scale=None, post_w=None, post_b=None, pre_w=None, dx_out=None, dh=None,
                      pre="layer", post="none", eps=1e-5, rows_per_group=None, mask=None):
    """Gradients by name, with `<name>_abs` the sums of the terms' magnitudes
    of every column sum (what its rounding scales with)."""
    T, C = (x_out if x_out is not None else dx_out).shape
    g = {}
    d = np.zeros((T, C)) if dx_out is None else dx_out
    if pre != "none":
        xh, r = _normed(x_out, pre, eps)
        g["dpre_w"], g["dpre_w_abs"] = (dh * xh).sum(0), np.abs(dh * xh).sum(0)
        g["dpre_b"], g["dpre_b_abs"] = dh.sum(0), np.abs(dh).sum(0)
        d = d + _normed_bwd(dh * _or(pre_w, 1.0), xh, r, pre)
    g["dx"] = d
    if y is None:
        return g
    yh, ry = _normed(y, post, eps)
    u = yh * _or(post_w, 1.0) + _or(post_b, 0.0)
    m, f, gt = _or(mask, 1.0), _rows(scale, T, rows_per_group), _or(gate, 1.0)
    g["dgate"] = d * m * f * u
    t = d * m * gt * u * np.ones((T, C))
    rpg = rows_per_group or T
    starts = np.arange(0, T, rpg) if T else np.zeros(0, int)
    g["dscale"] = np.stack([t[a:a + rpg].sum(0) for a in starts]) if T else np.zeros((0, C))
    g["dscale_abs"] = np.stack([np.abs(t[a:a + rpg]).sum(0) for a in starts]) if T else np.zeros((0, C))
    du = d * m * f * gt
    g["dpost_w"], g["dpost_w_abs"] = (du * yh).sum(0), np.abs(du * yh).sum(0)
    g["dpost_b"], g["dpost_b_abs"] = du.sum(0), np.abs(du).sum(0)
    g["dy"] = _normed_bwd(du * _or(post_w, 1.0), yh, ry, post)
    return g


# ------------------------------------------------------ differential attention
def window_rows(height, width, window):
    """Raster token numbers of each window x window cell of a map, cut at its edges."""
    out = []
    for y in range(0, height, window):
        for x in range(0, width, window):
            ys, xs = np.arange(y, min(y + window, height)), np.arange(x, min(x + window, width))
            out.append((ys[:, None] * width + xs[None]).reshape(-1))
    return out


def _softmax(s):
    """Row softmax and log-sum-exp; a row of -inf alone gives zeros and -inf."""
    m = s.max(1, keepdims=True) if s.shape[1] else np.full((s.shape[0], 1), -np.inf)
    p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = p.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(l > 0, np.where(np.isfinite(m), m, 0.0) + np.log(l), -np.inf)
    return p / np.where(l > 0, l, 1.0), lse[:, 0]


def _sequences(q, k, k_lens, causal, window, width):
    """(batch item, query rows, key rows, hidden mask or None) of every sequence."""
    B, Nq, Nk = q.shape[0], q.shape[1], k.shape[1]
    for b in range(B):
        if window:
            for r in window_rows(Nq // width, width, window):
                yield b, r, r, None
        else:
            n = Nk if k_lens is None else int(min(max(k_lens[b], 0), Nk))
            hide = np.arange(n)[None] > np.arange(Nq)[:, None] + n - Nq if causal else None
            yield b, np.arange(Nq), np.arange(n), hide


def diff_attention(q1, q2, k1, k2, v, lam, scale, k_lens=None, causal=False, window=0, width=0, dO=None):
    """Tensors [batch, tokens, heads, e], lam [q heads]. Returns a dict with o,
    o2 (the second map's output) and lse [2, batch, heads, tokens]; with dO
    also the gradients."""
    B, Nq, Hq, _ = q1.shape
    G = Hq // k1.shape[2]
    out = {"o": np.zeros((B, Nq, Hq, v.shape[3])), "lse": np.full((2, B, Hq, Nq), -np.inf)}
    out["o2"] = np.zeros_like(out["o"])
    if dO is not None:
        for n, t in (("dq1", q1), ("dq2", q2), ("dk1", k1), ("dk2", k2), ("dv", v)):
            out[n] = np.zeros(t.shape)
        out["dlam"] = np.zeros(Hq)
    for b, qr, kr, hide in _sequences(q1, k1, k_lens, causal, window, width):
        for h in range(Hq):
            g = h // G
            maps = []
            for i, (q, k) in enumerate(((q1, k1), (q2, k2))):
                s = q[b, qr, h] @ k[b, kr, g].T * scale
                if hide is not None:
                    s = np.where(hide, -np.inf, s)
                a, lse = _softmax(s)
                out["lse"][i, b, h, qr] = lse
                maps.append(a)
            vv = v[b, kr, g]
            o2 = maps[1] @ vv
            out["o2"][b, qr, h] = o2
            out["o"][b, qr, h] = maps[0] @ vv - lam[h] * o2
            if dO is None:
                continue
            do = dO[b, qr, h]
            dp = do @ vv.T
            out["dlam"][h] -= (do * o2).sum()
            out["dv"][b, kr, g] += (maps[0] - lam[h] * maps[1]).T @ do
            for a, q, k, nq, nk, f in ((maps[0], q1, k1, "dq1", "dk1", 1.0), (maps[1], q2, k2, "dq2", "dk2", -lam[h])):
                ds = f * scale * a * (dp - (a * dp).sum(1, keepdims=True))
                out[nq][b, qr, h] = ds @ k[b, kr, g]
                out[nk][b, kr, g] += ds.T @ q[b, qr, h]
    return out
