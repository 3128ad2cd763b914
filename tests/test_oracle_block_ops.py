"""Pins of the training-block oracle (CPU): the generator against published
test vectors, the norms against torch's fp64 functions, every gradient against
central differences."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as bo


def test_philox_matches_the_published_vectors():
    # the known answers published with the method's reference vectors (philox4x32, 10 rounds)
    f = 0xFFFFFFFF
    assert [hex(v) for v in bo.philox4x32_10([[0, 0, 0, 0]], (0, 0))[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    assert [hex(v) for v in bo.philox4x32_10([[f, f, f, f]], (f, f))[0]] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]


def test_dropout_factor_statistics_and_edges():
    n, p = 200_000, 0.1
    f = bo.dropout_factor(n, p, 7, 3)
    kept = (f > 0).mean()
    # kept share: binomial, five standard deviations
    assert abs(kept - (1 - round(p * 65536) / 65536)) < 5 * np.sqrt(0.09 / n)
    assert np.all(bo.dropout_factor(64, 0.0, 1, 1) == 1) and np.all(bo.dropout_factor(64, 1.0, 1, 1) == 0)
    assert np.array_equal(bo.dropout_factor(40, p, 7, 3), f[:40])
    assert np.array_equal(bo.dropout_factor(40, p, 7, 3, first=80), f[80:120])
    assert not np.array_equal(bo.dropout_factor(n, p, 7, 4), f)
    assert not np.array_equal(bo.dropout_factor(n, p, 8, 3), f)


def _diff(fn, v, g, eps=1e-6, picks=12, seed=0):
    """Largest difference of g from central differences of fn at a few entries of v."""
    r = np.random.default_rng(seed)
    worst = 0.0
    for _ in range(picks):
        i = tuple(int(r.integers(n)) for n in v.shape)
        keep = v[i]
        v[i] = keep + eps
        a = fn()
        v[i] = keep - eps
        b = fn()
        v[i] = keep
        worst = max(worst, abs((a - b) / (2 * eps) - g[i]))
    return worst


@pytest.mark.parametrize("pre,post,gated", [("layer", "layer", True), ("rms", "rms", True), ("layer", "none", False),
                                            ("none", "rms", True), ("rms", "layer", False)])
def test_residual_norm_gradients_match_differences(pre, post, gated):
    r = np.random.default_rng(1)
    T, C, rpg = 7, 12, 3
    a = {"x": r.normal(size=(T, C)), "y": r.normal(size=(T, C)), "scale": r.normal(size=(3, C))}
    if gated:
        a["gate"] = r.normal(size=(T, C))
    for n, kind in (("post", post), ("pre", pre)):
        if kind != "none":
            a[n + "_w"], a[n + "_b"] = r.normal(size=C), r.normal(size=C)
    mask = bo.dropout_factor(T * C, 0.3, 5, 9).reshape(T, C)
    kw = dict(pre=pre, post=post, rows_per_group=rpg, mask=mask)
    dx_out, dh = r.normal(size=(T, C)), r.normal(size=(T, C))

    def loss():
        x1, h = bo.residual_norm(a["x"], a["y"], *(a.get(k) for k in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")), **kw)
        return (x1 * dx_out).sum() + ((h * dh).sum() if h is not None else 0.0)

    x1, _ = bo.residual_norm(a["x"], a["y"], *(a.get(k) for k in ("gate", "scale", "post_w", "post_b", "pre_w", "pre_b")), **kw)
    g = bo.residual_norm_bwd(x1, a["y"], *(a.get(k) for k in ("gate", "scale", "post_w", "post_b", "pre_w")), dx_out=dx_out,
                             dh=dh if pre != "none" else None, **kw)
    for k, v in a.items():
        # second-order term of a central difference at 1e-6 is below 1e-9; rounding of the loss 1e-14 / 1e-6
        assert _diff(loss, v, g["d" + k]) < 1e-6, k


def test_norms_match_torch():
    r = np.random.default_rng(2)
    x, w, b = r.normal(size=(5, 33)), r.normal(size=33), r.normal(size=33)
    t = torch.from_numpy
    _, h = bo.residual_norm(x, pre_w=w, pre_b=b, pre="layer")
    assert np.abs(h - torch.nn.functional.layer_norm(t(x), (33,), t(w), t(b), 1e-5).numpy()).max() < 1e-12
    _, h = bo.residual_norm(x, pre_w=w, pre="rms")
    assert np.abs(h - torch.nn.functional.rms_norm(t(x), (33,), t(w), 1e-5).numpy()).max() < 1e-12


@pytest.mark.parametrize("case", ["plain", "causal", "lens", "window"])
def test_diff_attention_gradients_match_differences(case):
    r = np.random.default_rng(3)
    B, Hk, G, d, dv = 2, 2, 2, 4, 6
    Nq, Nk = (35, 35) if case == "window" else ((5, 7) if case != "causal" else (6, 6))
    a = {"q1": r.normal(size=(B, Nq, Hk * G, d)), "q2": r.normal(size=(B, Nq, Hk * G, d)), "k1": r.normal(size=(B, Nk, Hk, d)),
         "k2": r.normal(size=(B, Nk, Hk, d)), "v": r.normal(size=(B, Nk, Hk, dv)), "lam": r.normal(size=Hk * G)}
    dO = r.normal(size=(B, Nq, Hk * G, dv))
    kw = {"scale": 0.5, "causal": case == "causal"}
    if case == "lens":
        kw["k_lens"] = np.array([0, 4])
    if case == "window":
        kw.update(window=3, width=7)
    g = bo.diff_attention(*a.values(), dO=dO, **kw)
    for k, v in a.items():
        assert _diff(lambda: (bo.diff_attention(*a.values(), **kw)["o"] * dO).sum(), v, g["d" + k], picks=6) < 1e-6, k


def test_diff_attention_is_the_difference_of_two_attentions():
    r = np.random.default_rng(4)
    q1, q2, k1, k2 = (r.normal(size=(1, 9, 2, 8)) for _ in range(4))
    v, lam = r.normal(size=(1, 9, 2, 10)), np.array([0.3, -0.7])
    t = lambda x: torch.from_numpy(x).transpose(1, 2)  # noqa: E731
    sdpa = torch.nn.functional.scaled_dot_product_attention
    ref = sdpa(t(q1), t(k1), t(v), is_causal=True) - torch.from_numpy(lam)[:, None, None] * sdpa(t(q2), t(k2), t(v), is_causal=True)
    got = bo.diff_attention(q1, q2, k1, k2, v, lam, 8 ** -0.5, causal=True)
    assert np.abs(got["o"] - ref.transpose(1, 2).numpy()).max() < 1e-12
    assert np.all(bo.diff_attention(q1, q2, k1, k2, v, lam, 1.0, k_lens=[0])["o"] == 0)
